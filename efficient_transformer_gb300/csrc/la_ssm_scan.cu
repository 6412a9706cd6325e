// la_ssm_scan.cu -- selective state space scan over prompts: the scan itself, and the sums of segments alone (forward, and
// in reverse for the gradient) that cut long sequences into pieces that run at once.
//
// The decay differs by channel, state and token, so there is no product for the tensor cores: a state costs 4 float
// operations and one ex2 a token.  A warp holds 32 / LPC channels, the LPC lanes of a channel SPT states each, in registers.
// A lane finds d, d x and the gate of OWN = 8 / LPC of every eight tokens (its "own"); they go to the channel's
// lanes by shuffles, and the lanes' sums of C h come back to the owner by exchanged halves (quad_sums), so nothing of it
// passes through shared memory.  Rows of x, dt, z, B and C come by asynchronous copies a few tiles ahead; B and C, which all
// warps of a block read, are widened to float32 once a block.  Outputs replace the x that their lane alone has
// read and leave as whole rows.
#include "la_ssm.cuh"

namespace la {
namespace {

enum Mode { kScan = 0, kSums = 1, kReverse = 2 };

constexpr int kWarps = 4, kThreads = kWarps * 32, kRows = 16, kAhead = 3, kStages = kAhead + 2;

constexpr int spt_of(int S) { return S <= 16 ? 4 : 8; }

template <typename T, int S, int MODE>
struct Shape {
    static constexpr int SPT = spt_of(S), LPC = S / SPT, CPW = 32 / LPC, CH = kWarps * CPW, OWN = 8 / LPC;
    static constexpr int V = 16 / (int)sizeof(T);                            // elements of a copy
    static constexpr int TENSORS = MODE == kSums ? 2 : 3, MATS = MODE == kScan ? 2 : 1;
    // (16 bytes of padding: the lanes' reads of four tokens' rows fall on different banks)
    static constexpr int ROW = CH * (int)sizeof(T) + 16, BROW = S * (int)sizeof(T);
    static constexpr int XBYTES = kRows * ROW, BBYTES = kRows * BROW;
    static constexpr int STAGE = TENSORS * XBYTES + MATS * BBYTES;
    static constexpr int WIDE = kRows * MATS * S;                            // floats of a tile's B and C
    static constexpr int SMEM = kStages * STAGE + 2 * WIDE * 4;
};

template <typename T, int S, int MODE>
__global__ void __launch_bounds__(kThreads) k_ssm_scan(SsmParams p) {
    using H = Shape<T, S, MODE>;
    constexpr int SPT = H::SPT, LPC = H::LPC, CH = H::CH, OWN = H::OWN, V = H::V, TENSORS = H::TENSORS, MATS = H::MATS;
    constexpr int PAIRS = SPT / 2;
    extern __shared__ __align__(16) unsigned char smem[];
    float *wide = reinterpret_cast<float *>(smem + kStages * H::STAGE);
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane % LPC;
    const int tiles = (p.Eg + CH - 1) / CH;
    unsigned idx = blockIdx.x;
    const int ct = idx % tiles;
    idx /= tiles;
    const int grp = idx % p.G;
    idx /= p.G;
    const int nsegs = MODE == kScan ? p.nseg : p.nseg - 1;                   // segments of this launch
    const int seg = idx % nsegs + (MODE == kReverse), b = idx / nsegs;
    const int c0 = ct * CH, left = min(CH, p.Eg - c0);                       // the block's channels of its group
    const int mine = warp * H::CPW + lane / LPC;
    const bool there = mine < left;
    const int e = grp * p.Eg + c0 + (there ? mine : 0);
    const int t0 = seg * p.seg_len, t1 = min(t0 + p.seg_len, p.N);
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.N) : p.N;
    const int te = min(t1, len), nt = te > t0 ? (te - t0 + kRows - 1) / kRows : 0;

    auto row = [&](const void *base, const Strides &st) {
        return static_cast<const T *>(base) + b * st.b + (long long)t0 * st.n + grp * p.Eg + c0;
    };
    const T *src[3] = {row(MODE == kReverse ? p.g : p.x, MODE == kReverse ? p.sg : p.sx), row(p.dt, p.sdt), row(p.z, p.sz)};
    const long long step[3] = {MODE == kReverse ? p.sg.n : p.sx.n, p.sdt.n, p.sz.n};
    const T *mat[2];
    long long mstep[2];
    {
        const T *mB = static_cast<const T *>(p.B) + b * p.sB.b + (long long)t0 * p.sB.n + grp * p.sB.h;
        const T *mC = static_cast<const T *>(p.C) + b * p.sC.b + (long long)t0 * p.sC.n + grp * p.sC.h;
        mat[0] = MODE == kReverse ? mC : mB;
        mstep[0] = MODE == kReverse ? p.sC.n : p.sB.n;
        mat[1] = mC;
        mstep[1] = p.sC.n;
    }
    const bool gated = p.z != nullptr;

    // tile `i` of the order of work (in reverse: the last first) to its stage; rows past te and channels past the group: zeros
    auto place = [&](int i) { return MODE == kReverse ? nt - 1 - i : i; };
    auto load = [&](int i) {
        if (i < nt) {
            unsigned char *st = smem + (i % kStages) * H::STAGE;
            const int first = place(i) * kRows;
            constexpr int XV = CH / V, PER = kRows * XV;
#pragma unroll
            for (int k = 0; k < TENSORS; ++k) {
                if (k == 2 && !gated) break;
                for (int v = tid; v < PER; v += kThreads) {
                    const int t = v / XV, c = v % XV * V;
                    const bool in = t0 + first + t < te && c < left;
                    copy_async<16>(st + k * H::XBYTES + t * H::ROW + c * (int)sizeof(T),
                                   in ? src[k] + (long long)(first + t) * step[k] + c : src[k], in);
                }
            }
            constexpr int BV = S / V, BPER = kRows * BV;
#pragma unroll
            for (int k = 0; k < MATS; ++k)
                for (int v = tid; v < BPER; v += kThreads) {
                    const int t = v / BV, c = v % BV * V;
                    const bool in = t0 + first + t < te;
                    copy_async<16>(st + TENSORS * H::XBYTES + k * H::BBYTES + v * 16,
                                   in ? mat[k] + (long long)(first + t) * mstep[k] + c : mat[k], in);
                }
        }
        copy_commit();
    };
    // B and C of a tile as float32, [row][B states, C states]
    auto widen = [&](int i) {
        if (i >= nt) return;
        const unsigned char *st = smem + (i % kStages) * H::STAGE + TENSORS * H::XBYTES;
        float *to = wide + (i & 1) * H::WIDE;
        constexpr int BV = S / V, BPER = kRows * BV;
#pragma unroll
        for (int k = 0; k < MATS; ++k)
            for (int v = tid; v < BPER; v += kThreads)
                widen16(to + v / BV * (MATS * S) + k * S + v % BV * V, reinterpret_cast<const T *>(st + k * H::BBYTES + v * 16));
    };

#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(i);

    F2 A[PAIRS], h[PAIRS];
    const float bias = p.dt_bias ? p.dt_bias[e] : 0.f, skip = MODE == kScan && p.skip ? p.skip[e] : 0.f;
    {
        const float *a = p.A + (size_t)e * S + r * SPT;
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            A[i] = F2{a[2 * i] * kLog2e, a[2 * i + 1] * kLog2e};
            h[i] = f2(0.f);
        }
    }
    auto states = [&](const float *base, size_t block) { return base + (block * p.E + e) * S + r * SPT; };
    auto take = [&](const float *from) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) h[i] = *reinterpret_cast<const F2 *>(from + 2 * i);
    };
    auto put = [&](float *to) {
#pragma unroll
        for (int i = 0; i < SPT / 4; ++i)
            *reinterpret_cast<float4 *>(to + 4 * i) = make_float4(h[2 * i].x, h[2 * i].y, h[2 * i + 1].x, h[2 * i + 1].y);
    };
    // The start.  Segment 0's sum holds the initial state, so that only it is read besides the first segment itself, which
    // takes its copy in the last slot: the final state may replace the initial one at any time.
    if (MODE == kScan && p.nseg > 1) {
        const size_t w0 = (size_t)b * p.nseg;
        if (seg == 0) {
            if (p.init) take(states(p.seg_state, w0 + p.nseg - 1));
        } else {
            take(states(p.seg_state, w0));
            for (int j = 1; j < seg; ++j) {
                const float d = p.seg_d[(w0 + j) * p.E + e];
                const float *from = states(p.seg_state, w0 + j);
#pragma unroll
                for (int i = 0; i < PAIRS; ++i)
                    h[i] = fma2(ex22(mul2(f2(d), A[i])), h[i], *reinterpret_cast<const F2 *>(from + 2 * i));
            }
        }
    } else if (MODE != kReverse && seg == 0 && p.init) {
        take(states(p.init, b));
        if (MODE == kSums && there) put(const_cast<float *>(states(p.seg_state, (size_t)b * p.nseg + p.nseg - 1)));
    }
    float dsum = 0.f;

    // Every tile: the copies of the next one have come, whole (barrier); the last one's outputs leave; another is asked
    // for, into the stage that was emptied before the barrier; the next one's B and C are widened; this one is worked on.
    auto leave = [&](int i) {
        if (MODE != kScan || !p.out || i < 0) return;
        const unsigned char *st = smem + (i % kStages) * H::STAGE;
        constexpr int XV = CH / V, PER = kRows * XV;
        T *out = static_cast<T *>(p.out) + ((long long)b * p.N + t0 + (long long)i * kRows) * p.E + grp * p.Eg + c0;
        for (int v = tid; v < PER; v += kThreads) {
            const int t = v / XV, c = v % XV * V;
            if (t0 + i * kRows + t < te && c < left)
                *reinterpret_cast<uint4 *>(out + (long long)t * p.E + c) = *reinterpret_cast<const uint4 *>(st + t * H::ROW + c * (int)sizeof(T));
        }
    };
    copy_wait<kAhead - 1>();
    __syncthreads();
    widen(0);
    for (int i = 0; i < nt; ++i) {
        copy_wait<kAhead - 2>();
        __syncthreads();
        leave(i - 1);
        load(i + kAhead);
        widen(i + 1);
        unsigned char *st = smem + (i % kStages) * H::STAGE;
        const float *bc = wide + (i & 1) * H::WIDE + r * SPT;
        const int first = place(i) * kRows;
#pragma unroll 1
        for (int q = 0; q < kRows / 8; ++q) {
            const int c8 = MODE == kReverse ? kRows - 8 - q * 8 : q * 8;     // the eight tokens' place in the tile
            if (MODE == kScan && p.kept && there && t0 + first + c8 < te)
                put(const_cast<float *>(states(p.kept, (size_t)b * ((p.N + kSsmTile - 1) / kSsmTile) + (t0 + first + c8) / kSsmTile)));
            float d[OWN], u[OWN], x[OWN];
#pragma unroll
            for (int o = 0; o < OWN; ++o) {
                const int t = c8 + r * OWN + o;
                const unsigned char *at = st + t * H::ROW + mine * (int)sizeof(T);
                x[o] = to_f32(*reinterpret_cast<const T *>(at));
                const float v = to_f32(*reinterpret_cast<const T *>(at + H::XBYTES)) + bias;
                float ev;
                const float sp = p.softplus ? softplus(v, ev) : v;
                d[o] = t0 + first + t < te ? sp : 0.f;                       // past the length: h stays as it is
                if (MODE == kReverse) {
                    float gz = 1.f;
                    if (gated) {
                        const float z = to_f32(*reinterpret_cast<const T *>(at + 2 * H::XBYTES));
                        gz = z * sigmoid(z);
                    }
                    u[o] = x[o] * gz;                                        // the gradient of y
                } else {
                    u[o] = d[o] * x[o];
                }
                if (MODE != kScan) dsum += d[o];
            }
            float y[8];
#pragma unroll
            for (int jj = 0; jj < 8; ++jj) {
                const int j = MODE == kReverse ? 7 - jj : jj;
                const F2 dj = f2(__shfl_sync(0xffffffffu, d[j % OWN], j / OWN, LPC));
                const F2 uj = f2(__shfl_sync(0xffffffffu, u[j % OWN], j / OWN, LPC));
                const float *at = bc + (c8 + j) * (MATS * S);
                F2 acc = f2(0.f);
#pragma unroll
                for (int i4 = 0; i4 < SPT / 4; ++i4) {
                    const float4 m = *reinterpret_cast<const float4 *>(at + 4 * i4);
                    const F2 m2[2] = {F2{m.x, m.y}, F2{m.z, m.w}};
                    float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (MODE == kScan) c = *reinterpret_cast<const float4 *>(at + S + 4 * i4);
                    const F2 cc[2] = {F2{c.x, c.y}, F2{c.z, c.w}};
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        F2 &hk = h[2 * i4 + k];
                        const F2 a = ex22(mul2(dj, A[2 * i4 + k]));
                        if (MODE == kReverse) {
                            hk = mul2(a, fma2(uj, m2[k], hk));
                        } else {
                            hk = fma2(a, hk, mul2(uj, m2[k]));
                            if (MODE == kScan) acc = fma2(cc[k], hk, acc);
                        }
                    }
                }
                y[j] = acc.x + acc.y;
            }
            if (MODE == kScan) {
                quad_sums<LPC>(y, lane);
#pragma unroll
                for (int o = 0; o < OWN; ++o) {
                    unsigned char *at = st + (c8 + r * OWN + o) * H::ROW + mine * (int)sizeof(T);
                    float w = fmaf(skip, x[o], y[o]);
                    if (gated) {
                        const float z = to_f32(*reinterpret_cast<const T *>(at + 2 * H::XBYTES));
                        w *= z * sigmoid(z);
                    }
                    *reinterpret_cast<T *>(at) = from_f32<T>(w);
                }
            }
        }
    }
    if (MODE != kScan) {
        // the segment alone: its last state (in reverse: the gradient of the state before it) and its sum of d
#pragma unroll
        for (int m = 1; m < LPC; m <<= 1) dsum += __shfl_xor_sync(0xffffffffu, dsum, m);
        if (there) {
            const size_t w = (size_t)b * p.nseg + seg;
            put(const_cast<float *>(states(p.seg_state, w)));
            if (r == 0) p.seg_d[w * p.E + e] = dsum;
        }
        return;
    }
    if (p.fin && seg == p.nseg - 1 && there) put(const_cast<float *>(states(p.fin, b)));
    if (!p.out) return;
    __syncthreads();
    leave(nt - 1);
    // rows past the length
    T *out = static_cast<T *>(p.out) + (long long)b * p.N * p.E + grp * p.Eg + c0;
    constexpr int XV = CH / V;
    const int z0 = max(te, t0);
    for (long long v = tid; v < (long long)(t1 - z0) * XV; v += kThreads) {
        const int c = (int)(v % XV) * V;
        if (c < left) *reinterpret_cast<uint4 *>(out + (z0 + v / XV) * p.E + c) = make_uint4(0, 0, 0, 0);
    }
}

template <typename T, int S, int MODE>
cudaError_t launch(const SsmParams &p, cudaStream_t s) {
    using H = Shape<T, S, MODE>;
    TraceScope tr(MODE == kScan ? "ssm_scan" : MODE == kSums ? "ssm_sums" : "ssm_reverse_sums", s);
    auto kern = k_ssm_scan<T, S, MODE>;
    if (H::SMEM > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, H::SMEM);
        if (e != cudaSuccess) return e;
    }
    const long long blocks = (long long)((p.Eg + H::CH - 1) / H::CH) * p.G * p.nB * (MODE == kScan ? p.nseg : p.nseg - 1);
    return launch_pdl(kern, dim3((unsigned)blocks), dim3(kThreads), H::SMEM, s, p);
}

template <int MODE>
cudaError_t by_shape(const SsmParams &p, la_dtype dt, cudaStream_t s) {
    if (dt == LA_BF16) {
        if (p.S == 8) return launch<__nv_bfloat16, 8, MODE>(p, s);
        if (p.S == 16) return launch<__nv_bfloat16, 16, MODE>(p, s);
        if (p.S == 32) return launch<__nv_bfloat16, 32, MODE>(p, s);
        return launch<__nv_bfloat16, 64, MODE>(p, s);
    }
    if (p.S == 8) return launch<float, 8, MODE>(p, s);
    if (p.S == 16) return launch<float, 16, MODE>(p, s);
    if (p.S == 32) return launch<float, 32, MODE>(p, s);
    return launch<float, 64, MODE>(p, s);
}

}  // namespace

int ssm_scan_channels(int S) { return kWarps * 32 / (S / spt_of(S)); }

cudaError_t ssm_scan(const SsmParams &p, la_dtype dt, cudaStream_t s) { return by_shape<kScan>(p, dt, s); }

cudaError_t ssm_segments(const SsmParams &p, la_dtype dt, bool reverse, cudaStream_t s) {
    return reverse ? by_shape<kReverse>(p, dt, s) : by_shape<kSums>(p, dt, s);
}

}  // namespace la
