// la_ssm_grad.cu -- gradient of the selective state space scan.
//
// With a_t = exp(d_t A), u_t = d_t x_t, dy_t the gradient of y (grad_out times the gate) and G_t that of h_t,
//
//   G_t = C_t dy_t + P_t,   P_(t-1) = a_t G_t,   q_t = P_(t-1) h_(t-1)
//   dB_t = sum_e G u,  dC_t = sum_e dy h,  du = sum_s G B,  dA = sum_t q d,  dd = sum_s q A + x du
//   dx = d du + skip dy,  ddt = dd sigmoid(v),  dz = grad_out y (z sigmoid(z))',  dskip = sum dy x
//
// 12 float operations and one ex2 a state and token: h is found again from the state that the scan kept for every
// eight tokens, in registers, with a beside it; then the eight tokens are walked back.  Layout as in the scan: the LPC lanes of
// a channel hold 4 states each, a lane prepares its own tokens, sums over states come by exchanged halves.  The sums over
// channels (dB, dC) would cost more than all the rest if each token's were exchanged, so a warp takes K channel groups
// one after the other for the same eight tokens and adds up in 64 registers; only then are its lanes' sums exchanged, the warps'
// added in shared memory, and the block's written as one part.  P and dA wait in shared memory meanwhile.
#include "la_ssm.cuh"

namespace la {
namespace {

constexpr int kAhead = 2, kStages = kAhead + 2;

constexpr int warps_of(int S) { return S == 64 ? 8 : 4; }
// (128 channels a block; 64 states of float32 rows: 64, what shared memory holds)
constexpr int groups_of(int S, int bytes) { return S == 8 ? 2 : S == 16 || (S == 64 && bytes == 4) ? 4 : 8; }

template <typename T, int S>
struct Shape {
    static constexpr int LPC = S / 4, CPW = 32 / LPC, NW = warps_of(S), THREADS = NW * 32, OWN = LPC < 8 ? 8 / LPC : 1;
    static constexpr int CHK = NW * CPW, K = groups_of(S, (int)sizeof(T)), CH = CHK * K;
    static constexpr int V = 16 / (int)sizeof(T);
    static constexpr int ROW = CHK * (int)sizeof(T) + 16, XBYTES = K * 8 * ROW, BBYTES = 8 * S * (int)sizeof(T);
    static constexpr int STAGE = 4 * XBYTES + 2 * BBYTES;                  // x, dt, z, g [K][8][CHK]; B, C [8][S]
    static constexpr int WIDE = 8 * 2 * S;                                 // floats: B and C of a tile; a warp's dB and dC
    static constexpr int KEEP = K * THREADS;                               // float4 each: P, dA; float2: dskip, ddt_bias
    static constexpr int OFF_WIDE = kStages * STAGE, OFF_P = OFF_WIDE + 2 * WIDE * 4, OFF_A = OFF_P + KEEP * 16,
                         OFF_E = OFF_A + KEEP * 16, OFF_RED = OFF_E + KEEP * 8, SMEM = OFF_RED + 2 * NW * WIDE * 4;
    static_assert(SMEM <= 227 * 1024, "shared memory of a block");
};

template <typename T, int S>
__global__ void __launch_bounds__(Shape<T, S>::THREADS, S == 64 ? 1 : 3) k_ssm_grad(SsmParams p) {
    using H = Shape<T, S>;
    constexpr int LPC = H::LPC, OWN = H::OWN, V = H::V, CHK = H::CHK, TH = H::THREADS;
    extern __shared__ __align__(16) unsigned char smem[];
    float *wide = reinterpret_cast<float *>(smem + H::OFF_WIDE);
    float4 *keep_P = reinterpret_cast<float4 *>(smem + H::OFF_P), *keep_A = reinterpret_cast<float4 *>(smem + H::OFF_A);
    float2 *keep_e = reinterpret_cast<float2 *>(smem + H::OFF_E);
    float *red = reinterpret_cast<float *>(smem + H::OFF_RED);
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane % LPC, mine = warp * H::CPW + lane / LPC;
    const int blocks = (p.Eg + H::CH - 1) / H::CH;
    unsigned idx = blockIdx.x;
    const int cb = idx % blocks;
    idx /= blocks;
    const int grp = idx % p.G;
    idx /= p.G;
    const int seg = idx % p.nseg, b = idx / p.nseg;
    const int c0 = cb * H::CH, left = min(H::CH, p.Eg - c0), nk = (left + CHK - 1) / CHK;
    const int e0 = grp * p.Eg + c0;
    const int t0 = seg * p.seg_len, t1 = min(t0 + p.seg_len, p.N);
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.N) : p.N;
    const int te = min(t1, len), nt = te > t0 ? (te - t0 + 7) / 8 : 0;
    const bool gated = p.z != nullptr;

    auto row = [&](const void *base, const Strides &st) {
        return static_cast<const T *>(base) + b * st.b + (long long)t0 * st.n + e0;
    };
    const T *src[4] = {row(p.x, p.sx), row(p.dt, p.sdt), row(p.z, p.sz), row(p.g, p.sg)};
    const long long step[4] = {p.sx.n, p.sdt.n, p.sz.n, p.sg.n};
    const T *mat[2] = {static_cast<const T *>(p.B) + b * p.sB.b + (long long)t0 * p.sB.n + grp * p.sB.h,
                       static_cast<const T *>(p.C) + b * p.sC.b + (long long)t0 * p.sC.n + grp * p.sC.h};
    const long long mstep[2] = {p.sB.n, p.sC.n};

    // tiles go from the last to the first: the i-th is tile nt - 1 - i
    auto load = [&](int i) {
        if (i < nt) {
            unsigned char *st = smem + (i % kStages) * H::STAGE;
            const int first = (nt - 1 - i) * 8;
            constexpr int XV = CHK / V, PER = H::K * 8 * XV;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if (k == 2 && !gated) continue;
                for (int v = tid; v < PER; v += TH) {
                    const int t = v / XV % 8, kk = v / (8 * XV), c = kk * CHK + v % XV * V;
                    const bool in = t0 + first + t < te && c < left;
                    copy_async<16>(st + k * H::XBYTES + (kk * 8 + t) * H::ROW + v % XV * 16,
                                   in ? src[k] + (long long)(first + t) * step[k] + c : src[k], in);
                }
            }
            constexpr int BV = S / V, BPER = 8 * BV;
#pragma unroll
            for (int k = 0; k < 2; ++k)
                for (int v = tid; v < BPER; v += TH) {
                    const int t = v / BV, c = v % BV * V;
                    const bool in = t0 + first + t < te;
                    copy_async<16>(st + 4 * H::XBYTES + k * H::BBYTES + v * 16,
                                   in ? mat[k] + (long long)(first + t) * mstep[k] + c : mat[k], in);
                }
        }
        copy_commit();
    };
    auto widen = [&](int i) {
        if (i >= nt) return;
        const unsigned char *st = smem + (i % kStages) * H::STAGE + 4 * H::XBYTES;
        float *to = wide + (i & 1) * H::WIDE;
        constexpr int BV = S / V, BPER = 8 * BV;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            for (int v = tid; v < BPER; v += TH)
                widen16(to + v / BV * (2 * S) + k * S + v % BV * V, reinterpret_cast<const T *>(st + k * H::BBYTES + v * 16));
    };
    // what a tile leaves behind: rows of dx, ddt and dz (in the places of x, dt and z), and its part of dB and dC
    auto leave = [&](int i) {
        if (i < 0) return;
        const unsigned char *st = smem + (i % kStages) * H::STAGE;
        const int first = t0 + (nt - 1 - i) * 8;
        constexpr int XV = CHK / V, PER = H::K * 8 * XV;
        T *const to[3] = {static_cast<T *>(p.dx), static_cast<T *>(p.ddt), static_cast<T *>(p.dz)};
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (k == 2 && !gated) continue;
            T *out = to[k] + ((long long)b * p.N + first) * p.E + e0;
            for (int v = tid; v < PER; v += TH) {
                const int t = v / XV % 8, kk = v / (8 * XV), c = kk * CHK + v % XV * V;
                if (first + t < te && c < left)
                    *reinterpret_cast<uint4 *>(out + (long long)t * p.E + c) =
                        *reinterpret_cast<const uint4 *>(st + k * H::XBYTES + (kk * 8 + t) * H::ROW + v % XV * 16);
            }
        }
        const float *from = red + (i & 1) * H::NW * H::WIDE;
        float *part = p.part_bc + (((size_t)(grp * blocks + cb) * p.nB + b) * p.N + first) * (2 * S);
        for (int v = tid; v < H::WIDE; v += TH) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < H::NW; ++w) sum += from[w * H::WIDE + v];
            if (first + v / (2 * S) < te) part[v] = sum;
        }
    };

#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(i);

    // P of the segment's end: the final state's gradient through the later segments
#pragma unroll 1
    for (int k = 0; k < nk; ++k) {
        const int c = k * CHK + mine;
        const bool there = c < left;
        const size_t e = e0 + (there ? c : 0);
        const float4 A = *reinterpret_cast<const float4 *>(p.A + e * S + 4 * r);
        float4 P = p.dfinal && there ? *reinterpret_cast<const float4 *>(p.dfinal + ((size_t)b * p.E + e) * S + 4 * r)
                            : make_float4(0.f, 0.f, 0.f, 0.f);
        for (int j = p.nseg - 1; j > seg; --j) {
            const size_t w = ((size_t)b * p.nseg + j) * p.E + e;
            const float d = p.seg_d[w] * kLog2e;
            const float4 R = there ? *reinterpret_cast<const float4 *>(p.seg_state + w * S + 4 * r) : P;
            P = make_float4(fmaf(ex2(d * A.x), P.x, R.x), fmaf(ex2(d * A.y), P.y, R.y), fmaf(ex2(d * A.z), P.z, R.z),
                            fmaf(ex2(d * A.w), P.w, R.w));
        }
        keep_P[k * TH + tid] = P;
        keep_A[k * TH + tid] = make_float4(0.f, 0.f, 0.f, 0.f);
        keep_e[k * TH + tid] = make_float2(0.f, 0.f);
    }

    copy_wait<kAhead - 1>();
    __syncthreads();
    widen(0);
    const size_t kept0 = (size_t)b * ((p.N + kSsmTile - 1) / kSsmTile);
    auto kept = [&](int i, int k) {
        const int c = k * CHK + mine;
        const size_t w = (kept0 + t0 / 8 + nt - 1 - i) * p.E + e0 + c;
        return c < left ? *reinterpret_cast<const float4 *>(p.kept + w * S + 4 * r) : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    float4 h_next = make_float4(0.f, 0.f, 0.f, 0.f);
    if (nt > 0) h_next = kept(0, 0);
    for (int i = 0; i < nt; ++i) {
        copy_wait<kAhead - 2>();
        __syncthreads();
        leave(i - 1);
        load(i + kAhead);
        widen(i + 1);
        unsigned char *st = smem + (i % kStages) * H::STAGE;
        const float *bc = wide + (i & 1) * H::WIDE + 4 * r;
        const int first = t0 + (nt - 1 - i) * 8;
        F2 accB[8][2], accC[8][2];
#pragma unroll
        for (int j = 0; j < 8; ++j)
#pragma unroll
            for (int m = 0; m < 2; ++m) accB[j][m] = accC[j][m] = f2(0.f);
#pragma unroll 1
        for (int k = 0; k < nk; ++k) {
            const int c = k * CHK + mine;
            const bool there = c < left;
            const int e = e0 + (there ? c : 0);
            const float4 h4 = h_next;
            if (k + 1 < nk) h_next = kept(i, k + 1);
            else if (i + 1 < nt) h_next = kept(i + 1, 0);
            const float4 A4 = *reinterpret_cast<const float4 *>(p.A + (size_t)e * S + 4 * r);
            const F2 A[2] = {F2{A4.x * kLog2e, A4.y * kLog2e}, F2{A4.z * kLog2e, A4.w * kLog2e}};
            const float bias = p.dt_bias ? p.dt_bias[e] : 0.f, skip = p.skip ? p.skip[e] : 0.f;
            // the lane's own tokens
            float x[OWN], d[OWN], u[OWN], dy[OWN], slope[OWN], gz[OWN];
            unsigned char *at0 = st + (k * 8 + (LPC == 16 ? r % 8 : r * OWN)) * H::ROW + mine * (int)sizeof(T);
            const int own0 = first + (LPC == 16 ? r % 8 : r * OWN);
#pragma unroll
            for (int o = 0; o < OWN; ++o) {
                const unsigned char *at = at0 + o * H::ROW;
                auto get = [&](int m) { return to_f32(*reinterpret_cast<const T *>(at + m * H::XBYTES)); };
                x[o] = get(0);
                const float v = get(1) + bias, g = get(3);
                float sp = v;
                slope[o] = 1.f;
                if (p.softplus) {
                    float ev;
                    sp = softplus(v, ev);
                    const float s1 = rcp(1.f + ev);
                    slope[o] = v >= 0.f ? s1 : ev * s1;
                }
                const bool in = own0 + o < te;
                d[o] = in ? sp : 0.f;
                u[o] = d[o] * x[o];
                dy[o] = g;
                gz[o] = 0.f;
                if (gated) {
                    const float z = get(2), sz = sigmoid(z);
                    dy[o] = g * (z * sz);
                    gz[o] = g * sz * fmaf(z, 1.f - sz, 1.f);
                }
            }
            auto all = [&](const float (&v)[OWN], int j) {   // token j's value, from the lane that owns it
                return __shfl_sync(0xffffffffu, v[j % OWN], j / OWN, LPC);
            };
            // forward: h after each token, a beside it
            F2 a[8][2], hs[8][2];
            {
                F2 h[2] = {F2{h4.x, h4.y}, F2{h4.z, h4.w}};
                float y[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const F2 dj = f2(all(d, j)), uj = f2(all(u, j)), gj = f2(all(dy, j));
                    const float4 B4 = *reinterpret_cast<const float4 *>(bc + j * 2 * S), C4 = *reinterpret_cast<const float4 *>(bc + j * 2 * S + S);
                    const F2 Bj[2] = {F2{B4.x, B4.y}, F2{B4.z, B4.w}}, Cj[2] = {F2{C4.x, C4.y}, F2{C4.z, C4.w}};
                    F2 acc = f2(0.f);
#pragma unroll
                    for (int m = 0; m < 2; ++m) {
                        a[j][m] = ex22(mul2(dj, A[m]));
                        h[m] = fma2(a[j][m], h[m], mul2(uj, Bj[m]));
                        hs[j][m] = h[m];
                        accC[j][m] = fma2(gj, h[m], accC[j][m]);
                        acc = fma2(Cj[m], h[m], acc);
                    }
                    y[j] = acc.x + acc.y;
                }
                if (gated) {
                    quad_sums<LPC>(y, lane);
#pragma unroll
                    for (int o = 0; o < OWN; ++o)
                        if (LPC < 16 || r < 8)
                            *reinterpret_cast<T *>(at0 + o * H::ROW + 2 * H::XBYTES) = from_f32<T>(gz[o] * fmaf(skip, x[o], y[o]));
                }
            }
            // and back
            float du[8], dq[8];
            const float4 P4 = keep_P[k * TH + tid], dA4 = keep_A[k * TH + tid];
            F2 P[2] = {F2{P4.x, P4.y}, F2{P4.z, P4.w}}, dA[2] = {F2{dA4.x, dA4.y}, F2{dA4.z, dA4.w}};
#pragma unroll
            for (int j = 7; j >= 0; --j) {
                const F2 dj = f2(all(d, j)), uj = f2(all(u, j)), gj = f2(all(dy, j));
                const float4 B4 = *reinterpret_cast<const float4 *>(bc + j * 2 * S), C4 = *reinterpret_cast<const float4 *>(bc + j * 2 * S + S);
                const F2 Bj[2] = {F2{B4.x, B4.y}, F2{B4.z, B4.w}}, Cj[2] = {F2{C4.x, C4.y}, F2{C4.z, C4.w}};
                F2 sb = f2(0.f), sq = f2(0.f);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const F2 before = j > 0 ? hs[j > 0 ? j - 1 : 0][m] : m == 0 ? F2{h4.x, h4.y} : F2{h4.z, h4.w};
                    const F2 G = fma2(Cj[m], gj, P[m]);
                    sb = fma2(G, Bj[m], sb);
                    accB[j][m] = fma2(G, uj, accB[j][m]);
                    P[m] = mul2(a[j][m], G);
                    const F2 q = mul2(P[m], before);
                    sq = fma2(q, A[m], sq);
                    dA[m] = fma2(q, dj, dA[m]);
                }
                du[j] = sb.x + sb.y;
                dq[j] = sq.x + sq.y;
            }
            keep_P[k * TH + tid] = make_float4(P[0].x, P[0].y, P[1].x, P[1].y);
            keep_A[k * TH + tid] = make_float4(dA[0].x, dA[0].y, dA[1].x, dA[1].y);
            quad_sums<LPC>(du, lane);
            quad_sums<LPC>(dq, lane);
            float2 es = keep_e[k * TH + tid];
#pragma unroll
            for (int o = 0; o < OWN; ++o) {
                const float dx = fmaf(d[o], du[o], skip * dy[o]);
                // (past the length: d, x and dy are zeros, the sums over states are not)
                const float ddt = own0 + o < te ? fmaf(x[o], du[o], kLn2 * dq[o]) * slope[o] : 0.f;
                es.x = fmaf(dy[o], x[o], es.x);
                es.y += ddt;
                if (LPC < 16 || r < 8) {
                    *reinterpret_cast<T *>(at0 + o * H::ROW) = from_f32<T>(dx);
                    *reinterpret_cast<T *>(at0 + o * H::ROW + H::XBYTES) = from_f32<T>(ddt);
                }
            }
            keep_e[k * TH + tid] = es;
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
        int base = 0, n = 64;
#pragma unroll
        for (int m = 16; m >= LPC; m >>= 1) {
            n >>= 1;
            const bool up = lane & m;
            base += up ? n : 0;
#pragma unroll
            for (int q = 0; q < 32; ++q)
                if (q < n) {
                    const float send = up ? v[q] : v[q + n], hold = up ? v[q + n] : v[q];
                    v[q] = hold + __shfl_xor_sync(0xffffffffu, send, m);
                }
        }
        constexpr int LEFT = 64 / H::CPW;   // values a lane is left with
        float *to = red + ((i & 1) * H::NW + warp) * H::WIDE + 4 * r;
#pragma unroll
        for (int q = 0; q < LEFT; q += 4) {
            if (LEFT >= 4) {
                const int w = base + q;
                *reinterpret_cast<float4 *>(to + (w / 8) * 2 * S + (w % 8 / 4) * S) = make_float4(v[q], v[q + 1], v[q + 2], v[q + 3]);
            }
        }
    }
    __syncthreads();
    leave(nt - 1);
    // rows past the length
    {
        constexpr int XV = H::CH / V;
        const int z0 = max(te, t0);
        T *const to[3] = {static_cast<T *>(p.dx), static_cast<T *>(p.ddt), static_cast<T *>(p.dz)};
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (k == 2 && !gated) continue;
            T *out = to[k] + (long long)b * p.N * p.E + e0;
            for (long long v = tid; v < (long long)(t1 - z0) * XV; v += TH) {
                const int c = (int)(v % XV) * V;
                if (c < left) *reinterpret_cast<uint4 *>(out + (z0 + v / XV) * p.E + c) = make_uint4(0, 0, 0, 0);
            }
        }
    }
#pragma unroll 1
    for (int k = 0; k < nk; ++k) {
        const int c = k * CHK + mine;
        const bool there = c < left;
        const size_t e = e0 + (there ? c : 0), w = (size_t)b * p.nseg + seg;
        float2 es = keep_e[k * TH + tid];
#pragma unroll
        for (int m = 1; m < (LPC == 16 ? 8 : LPC); m <<= 1) {
            es.x += __shfl_xor_sync(0xffffffffu, es.x, m);
            es.y += __shfl_xor_sync(0xffffffffu, es.y, m);
        }
        if (!there) continue;
        *reinterpret_cast<float4 *>(p.part_A + (w * p.E + e) * S + 4 * r) = keep_A[k * TH + tid];
        if (r == 0) {
            p.part_e[(w * 2) * p.E + e] = es.x;
            p.part_e[(w * 2 + 1) * p.E + e] = es.y;
        }
        if (p.dinit && seg == 0) *reinterpret_cast<float4 *>(p.dinit + ((size_t)b * p.E + e) * S + 4 * r) = keep_P[k * TH + tid];
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

int ssm_grad_channels(int S, la_dtype dt) { return warps_of(S) * (32 / (S / 4)) * groups_of(S, dt == LA_BF16 ? 2 : 4); }

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
