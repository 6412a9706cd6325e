// la_ssm_scan.cu -- selective state space scan over prompts: the scan itself, and the sums of segments alone (forward, and
// in reverse for the gradient) that cut long sequences into pieces that run at once.
//
// The decay differs by channel, state and token, so there is no product for the tensor cores: a state costs 4 float
// operations and one ex2 a token.  A warp holds 32 / LPC channels, the LPC lanes of a channel SPT states each, in registers.
// A lane finds d, d x and the gate of OWN = 8 / LPC of every eight tokens (its "own"); they go to the channel's
// lanes by shuffles, and the lanes' sums of C h come back to the owner by exchanged halves (part_sums), so nothing of it
// passes through shared memory.  Rows of x, dt, z, B and C come by asynchronous copies two tiles ahead; B and C, which all
// warps of a block read, are widened to float32 once a block.  Outputs replace the x that their lane alone has
// read and leave as whole rows.
//
// 65536 x 2048 x 16, bfloat16: 598 us for the scan, 392 for the sums of 18 of its 19 segments; 16 x 2048 x 4096 x 16 in one
// segment 598.  All pipes are near each other: of the scan's time issue slots 61 %, shared memory 66 %, float operations
// 49 %, ex2 42 %; the bytes alone would take a quarter (1.9 TB/s).  float32: 667 and 402.
#include "la_ssm.cuh"

namespace la {
namespace {

enum Mode { kScan = 0, kSums = 1, kReverse = 2 };

constexpr int kWarps = 4, kThreads = kWarps * 32, kRows = 16, kAhead = 2, kStages = kAhead + 3;

// States of a lane: 8, or 16 where a channel would be spread over more than four lanes.  (4 a lane make twice the warps, but
// share a channel's preparation, shuffles and sums among fewer states: a third more instructions, 4 x 4096 x 4096 x 16 420 us
// against 352.)
constexpr int spt_of(int S) { return S <= 32 ? 8 : 16; }

template <typename T, int S, int MODE>
struct Shape {
    static constexpr int SPT = spt_of(S), LPC = S / SPT, CPW = 32 / LPC, CH = kWarps * CPW, OWN = 8 / LPC;
    static constexpr int V = 16 / (int)sizeof(T);                            // elements of a copy
    static constexpr int TENSORS = MODE == kSums ? 2 : 3, MATS = MODE == kScan ? 2 : 1;
    // (16 bytes of padding: the lanes' reads of four tokens' rows fall on different banks)
    static constexpr int ROW = CH * (int)sizeof(T) + 16, BROW = S * (int)sizeof(T);
    static constexpr int XBYTES = kRows * ROW, BBYTES = kRows * BROW;
    static constexpr int STAGE = TENSORS * XBYTES + MATS * BBYTES;
    static constexpr int XV = CH / V, NX = kRows * XV, BV = S / V, NB = kRows * BV;   // copies of a row, of a tile
    static constexpr int COPIES = (TENSORS * NX + MATS * NB + kThreads - 1) / kThreads;
    static constexpr int WIDE = kRows * MATS * S;                            // floats of a tile's B and C
    static constexpr int SMEM = kStages * STAGE + 2 * WIDE * 4;
};

// (four blocks an SM where the sums fit 128 registers without spills)
template <typename T, int S, int MODE>
__global__ void __launch_bounds__(kThreads, MODE != kScan && (S == 16 || S == 32) ? 4 : 3) k_ssm_scan(SsmParams p) {
    using H = Shape<T, S, MODE>;
    constexpr int SPT = H::SPT, LPC = H::LPC, CPW = H::CPW, CH = H::CH, OWN = H::OWN, V = H::V, TENSORS = H::TENSORS, MATS = H::MATS;
    constexpr int PAIRS = SPT / 2, OP = OWN > 1 ? OWN / 2 : 1;               // pairs of own tokens (of one: it and itself)
    extern __shared__ __align__(16) unsigned char smem[];
    float *wide = reinterpret_cast<float *>(smem + kStages * H::STAGE);
    pdl_wait();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane / CPW, chan = lane % CPW;
    const int tiles = (p.Eg + CH - 1) / CH;
    unsigned idx = blockIdx.x;
    const int ct = idx % tiles;
    idx /= tiles;
    const int grp = idx % p.G;
    idx /= p.G;
    const int nsegs = MODE == kScan ? p.nseg : p.nseg - 1;                   // segments of this launch
    const int seg = idx % nsegs + (MODE == kReverse), b = idx / nsegs;
    const int c0 = ct * CH, left = min(CH, p.Eg - c0);                       // the block's channels of its group
    const int mine = warp * CPW + chan;
    const bool there = mine < left;
    const int e = grp * p.Eg + c0 + (there ? mine : 0);
    const int t0 = seg * p.seg_len, t1 = min(t0 + p.seg_len, p.N);
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.N) : p.N;
    const int te = min(t1, len), n = max(te - t0, 0), nt = (n + kRows - 1) / kRows;
    const bool gated = p.z != nullptr;

    // A thread's copies: the same place of every tile, a tile's step apart.  Tiles in the order of work (in reverse: the last
    // first); rows past te and channels past the group's: zeros.
    const T *from[H::COPIES];
    long long step[H::COPIES];
    int row[H::COPIES];
    unsigned to[H::COPIES];
#pragma unroll
    for (int k = 0; k < H::COPIES; ++k) {
        const int v = tid + k * kThreads;
        const void *base = p.x;
        Strides st = p.sx;
        int c;
        if (v < TENSORS * H::NX) {
            const int w = v % H::NX, m = v / H::NX;
            if (MODE == kReverse && m == 0) base = p.g, st = p.sg;
            if (m == 1) base = p.dt, st = p.sdt;
            if (m == 2) base = p.z, st = p.sz;
            row[k] = w / H::XV;
            c = w % H::XV * V;
            to[k] = m * H::XBYTES + row[k] * H::ROW + c * (int)sizeof(T);
            if (c >= left || !base) row[k] = 1 << 30;
            c += grp * p.Eg + c0;
        } else {
            const int u = v - TENSORS * H::NX, m = u / H::NB;
            const bool C = MODE == kReverse || m == 1;
            base = C ? p.C : p.B;
            st = C ? p.sC : p.sB;
            row[k] = u % H::NB / H::BV;
            c = u % H::BV * V;
            to[k] = TENSORS * H::XBYTES + u * 16;
            if (m >= MATS) row[k] = 1 << 30;
            base = static_cast<const T *>(base) + grp * st.h;
        }
        const long long first = t0 + (MODE == kReverse ? (nt - 1) * kRows : 0);
        from[k] = row[k] < kRows ? static_cast<const T *>(base) + b * st.b + (first + row[k]) * st.n + c : nullptr;
        step[k] = (MODE == kReverse ? -kRows : kRows) * st.n;
    }
    const T *const anchor = static_cast<const T *>(p.dt);
    auto load = [&](int i, int stage) {
        if (i < nt) {
            const int first = (MODE == kReverse ? nt - 1 - i : i) * kRows;
#pragma unroll
            for (int k = 0; k < H::COPIES; ++k) {
                const bool in = first + row[k] < n;
                if ((k + 1) * kThreads <= TENSORS * H::NX + MATS * H::NB || tid + k * kThreads < TENSORS * H::NX + MATS * H::NB)
                    copy_async(smem + stage * H::STAGE + to[k], in ? from[k] : anchor, in);
                from[k] += step[k];
            }
        }
        copy_commit();
    };
    // B and C of a tile as float32, [row][B states, C states]
    auto widen = [&](int i, int stage) {
        if (i >= nt) return;
        const unsigned char *st = smem + stage * H::STAGE + TENSORS * H::XBYTES;
        float *w = wide + (i & 1) * H::WIDE;
#pragma unroll
        for (int k = 0; k < (MATS * H::NB + kThreads - 1) / kThreads; ++k) {
            const int v = tid + k * kThreads;
            if (MATS * H::NB % kThreads == 0 || v < MATS * H::NB)
                widen16(w + v % H::NB / H::BV * (MATS * S) + v / H::NB * S + v % H::BV * V, reinterpret_cast<const T *>(st + v * 16));
        }
    };
    // the outputs of a tile, in the places of its x
    T *out = MODE == kScan && p.out ? static_cast<T *>(p.out) + ((long long)b * p.N + t0) * p.E + grp * p.Eg + c0 : nullptr;
    auto leave = [&](int i, int stage) {
        if (MODE != kScan || !out || i < 0) return;
        const unsigned char *st = smem + stage * H::STAGE;
#pragma unroll
        for (int k = 0; k < (H::NX + kThreads - 1) / kThreads; ++k) {
            const int v = tid + k * kThreads, t = v / H::XV, c = v % H::XV * V;
            if ((H::NX % kThreads == 0 || v < H::NX) && i * kRows + t < n && c < left)
                *reinterpret_cast<uint4 *>(out + (long long)(i * kRows + t) * p.E + c) =
                    *reinterpret_cast<const uint4 *>(st + t * H::ROW + c * (int)sizeof(T));
        }
    };

#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(i, i);

    F2 A[PAIRS], h[PAIRS];
    float slow;                                                              // the least |A|
    const float bias = p.dt_bias ? p.dt_bias[e] : 0.f, skip = MODE == kScan && p.skip ? p.skip[e] : 0.f;
    {
        const float *a = p.A + (size_t)e * S + r * SPT;
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            A[i] = F2{a[2 * i] * kLog2e, a[2 * i + 1] * kLog2e};
            h[i] = f2(0.f);
            const float least = fminf(fabsf(A[i].x), fabsf(A[i].y));
            slow = i == 0 ? least : fminf(slow, least);
        }
    }
    auto states = [&](const float *base, size_t block) { return base + (block * p.E + e) * S + r * SPT; };
    auto take = [&](const float *a) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) h[i] = *reinterpret_cast<const F2 *>(a + 2 * i);
    };
    auto put = [&](float *a) {
#pragma unroll
        for (int i = 0; i < SPT / 4; ++i)
            *reinterpret_cast<float4 *>(a + 4 * i) = make_float4(h[2 * i].x, h[2 * i].y, h[2 * i + 1].x, h[2 * i + 1].y);
    };
    // The start.  Segment 0's sum holds the initial state, so that only it is read besides the first segment itself, which
    // takes its copy in the last slot: the final state may replace the initial one at any time.
    if (MODE == kScan && p.nseg > 1) {
        const size_t w0 = (size_t)b * p.nseg;
        if (seg == 0) {
            if (p.init) take(states(p.seg_state, w0 + p.nseg - 1));
        } else {
            take(states(p.seg_state, w0));
#pragma unroll 4
            for (int j = 1; j < seg; ++j) {
                const float d = p.seg_d[(w0 + j) * p.E + e];
                const float *a = states(p.seg_state, w0 + j);
#pragma unroll
                for (int i = 0; i < PAIRS; ++i) {
                    const F2 sum = *reinterpret_cast<const F2 *>(a + 2 * i);
                    h[i] = F2{join(d, A[i].x, h[i].x, sum.x), join(d, A[i].y, h[i].y, sum.y)};
                }
            }
        }
    } else if (MODE != kReverse && seg == 0 && p.init) {
        take(states(p.init, b));
        if (MODE == kSums && there) put(const_cast<float *>(states(p.seg_state, (size_t)b * p.nseg + p.nseg - 1)));
    }
    // (states kept for the gradient: [tile][S / 4][E][4])
    float *kept = MODE == kScan && p.kept && there
                      ? p.kept + (((size_t)b * ((p.N + kSsmTile - 1) / kSsmTile) + t0 / kSsmTile) * S / 4 * p.E + e) * 4 +
                            (size_t)r * (SPT / 4) * p.E * 4
                      : nullptr;
    float dsum = 0.f;

    // Eight tokens at a time, in three parts that overlap: the next ones' steps are prepared and the last ones' sums and gates
    // are finished while these run through the states.  No branches between them (what a call does not have is selected
    // away), so that the compiler may interleave all three: a warp alone on its scheduler would wait for most of them.
    struct Own {
        F2 d[OP], u[OP], x[OP];
    };
    unsigned char *const mine0 = smem + r * OWN * H::ROW + mine * (int)sizeof(T);
    auto pair = [&](const unsigned char *at, int m, int o) {                 // own tokens 2 o and 2 o + 1 of tensor m
        const unsigned char *a = at + m * H::XBYTES + 2 * o * H::ROW;
        return F2{to_f32(*reinterpret_cast<const T *>(a)), to_f32(*reinterpret_cast<const T *>(a + (OWN > 1 ? H::ROW : 0)))};
    };
    const bool sp = p.softplus;
    auto gate = [&](const unsigned char *at, int o) {
        const F2 z = pair(at, 2, o), g = mul2(z, sigmoid(z));
        return F2{gated ? g.x : 1.f, gated ? g.y : 1.f};
    };
    auto prepare = [&](const unsigned char *at, int t, Own &w) {             // t: of the lane's first own token, from t0 on
#pragma unroll
        for (int o = 0; o < OP; ++o) {
            w.x[o] = pair(at, 0, o);
            const F2 v = add2(pair(at, 1, o), f2(bias));
            F2 ev;
            const F2 s = softplus(v, ev);
            // (past the length: h stays as it is)
            w.d[o] = F2{t + 2 * o < n ? (sp ? s.x : v.x) : 0.f, t + 2 * o + 1 < n ? (sp ? s.y : v.y) : 0.f};
            w.u[o] = MODE == kReverse ? mul2(w.x[o], gate(at, o)) : mul2(w.d[o], w.x[o]);   // (in reverse: the gradient of y)
        }
    };
    auto run = [&](const Own &w, const float *bc, float (&y)[8]) {           // bc: the tokens' B and C
        auto all = [&](const F2 (&v)[OP], int j) {                           // token j's value, from the lane that owns it
            const int o = j % OWN;
            return f2(__shfl_sync(0xffffffffu, o % 2 ? v[o / 2].y : v[o / 2].x, j / OWN * CPW + chan));
        };
        const F2 d0 = all(w.d, 0), tilt = tilt_of(d0.x * slow);
#pragma unroll
        for (int jj = 0; jj < 8; ++jj) {
            const int j = MODE == kReverse ? 7 - jj : jj;
            const F2 dj = j == 0 ? d0 : all(w.d, j), uj = all(w.u, j);
            const float *m4 = bc + j * (MATS * S);
            F2 acc;
#pragma unroll
            for (int i4 = 0; i4 < SPT / 4; ++i4) {
                const float4 m = *reinterpret_cast<const float4 *>(m4 + 4 * i4);
                const F2 m2[2] = {F2{m.x, m.y}, F2{m.z, m.w}};
                float4 c = make_float4(0.f, 0.f, 0.f, 0.f);
                if (MODE == kScan) c = *reinterpret_cast<const float4 *>(m4 + S + 4 * i4);
                const F2 cc[2] = {F2{c.x, c.y}, F2{c.z, c.w}};
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    F2 &hk = h[2 * i4 + k];
                    const F2 a = decay2(dj, A[2 * i4 + k], tilt);
                    if (MODE == kReverse) {
                        hk = mul2(a, fma2(uj, m2[k], hk));
                    } else {
                        hk = fma2(a, hk, mul2(uj, m2[k]));
                        if (MODE == kScan) acc = i4 + k == 0 ? mul2(cc[k], hk) : fma2(cc[k], hk, acc);
                    }
                }
            }
            if (MODE == kScan) y[j] = acc.x + acc.y;
        }
    };
    auto finish = [&](unsigned char *at, const Own &w, float (&y)[8]) {
        if (MODE != kScan) return;
        part_sums<LPC, 8>(y, lane);
#pragma unroll
        for (int o = 0; o < OP; ++o) {
            F2 v = fma2(f2(skip), w.x[o], F2{y[2 * o], OWN > 1 ? y[2 * o + 1] : y[2 * o]});
            v = mul2(v, gate(at, o));
            *reinterpret_cast<T *>(at + 2 * o * H::ROW) = from_f32<T>(v.x);
            if (OWN > 1) *reinterpret_cast<T *>(at + (2 * o + 1) * H::ROW) = from_f32<T>(v.y);
        }
    };
    auto keep = [&](bool in) {
        if (MODE != kScan) return;
        if (kept && in) {
#pragma unroll
            for (int k = 0; k < SPT / 4; ++k)
                *reinterpret_cast<float4 *>(kept + (size_t)k * p.E * 4) = make_float4(h[2 * k].x, h[2 * k].y, h[2 * k + 1].x, h[2 * k + 1].y);
            kept += (size_t)S * p.E;
        }
    };

    // Every tile: the copies of the next one have come, whole (barrier); the outputs of the one before the last leave; another
    // is asked for, into the stage that was emptied before the barrier; the next one's B and C are widened; this one is run.
    constexpr int C0 = MODE == kReverse ? 8 : 0, C1 = 8 - C0;                // the places of its first and second eight tokens
    static_assert(kRows == 16, "two times eight tokens a tile");
    copy_wait<kAhead - 1>();
    __syncthreads();
    widen(0, 0);
    int stage = 0;
    auto after = [](int s, int k) { return s + k >= kStages ? s + k - kStages : s + k; };
    Own own[2];
    float y[2][8];
    prepare(mine0 + C0 * H::ROW, (MODE == kReverse ? (nt - 1) * kRows : 0) + C0 + r * OWN, own[0]);
    own[1] = own[0];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[1][j] = 0.f;
    // (a sum of d counts what is run, not what is prepared)
    auto count = [&](const Own &w) {
        if constexpr (MODE != kScan) {
#pragma unroll
            for (int o = 0; o < OP; ++o) dsum += OWN > 1 ? w.d[o].x + w.d[o].y : w.d[o].x;
        }
    };
    for (int i = 0; i < nt; ++i) {
        copy_wait<kAhead - 2>();
        __syncthreads();
        leave(i - 2, after(stage, kStages - 2));
        load(i + kAhead, after(stage, kAhead));
        widen(i + 1, after(stage, 1));
        unsigned char *const at = mine0 + stage * H::STAGE, *const next = mine0 + after(stage, 1) * H::STAGE,
                      *const last = mine0 + after(stage, kStages - 1) * H::STAGE;
        const float *bc = wide + (i & 1) * H::WIDE + r * SPT;
        const int first = (MODE == kReverse ? nt - 1 - i : i) * kRows, then = first + (MODE == kReverse ? -kRows : kRows);
        stage = after(stage, 1);
        keep(first < n);
        count(own[0]);
        {
            Own w;
            prepare(at + C1 * H::ROW, first + C1 + r * OWN, w);
            run(own[0], bc + C0 * (MATS * S), y[0]);
            finish(last + C1 * H::ROW, own[1], y[1]);   // (before the first tile: into a stage that nothing reads)
            own[1] = w;
        }
        keep(first + 8 < n);
        count(own[1]);
        {
            Own w;
            prepare(next + C0 * H::ROW, then + C0 + r * OWN, w);
            run(own[1], bc + C1 * (MATS * S), y[1]);
            finish(at + C0 * H::ROW, own[0], y[0]);
            own[0] = w;
        }
    }
    finish(mine0 + after(stage, kStages - 1) * H::STAGE + C1 * H::ROW, own[1], y[1]);
    if (MODE != kScan) {
        // the segment alone: its last state (in reverse: the gradient of the state before it) and its sum of d
#pragma unroll
        for (int m = CPW; LPC > 1 && m < 32; m <<= 1) dsum += __shfl_xor_sync(0xffffffffu, dsum, m);
        if (there) {
            const size_t w = (size_t)b * p.nseg + seg;
            put(const_cast<float *>(states(p.seg_state, w)));
            if (r == 0) p.seg_d[w * p.E + e] = dsum;
        }
        return;
    }
    if (p.fin && seg == p.nseg - 1 && there) put(const_cast<float *>(states(p.fin, b)));
    if (!out) return;
    __syncthreads();
    leave(nt - 2, after(stage, kStages - 2));
    leave(nt - 1, after(stage, kStages - 1));
    // rows past the length
    for (long long v = (long long)n * H::XV + tid; v < (long long)(t1 - t0) * H::XV; v += kThreads) {
        const int c = (int)(v % H::XV) * V;
        if (c < left) *reinterpret_cast<uint4 *>(out + (v / H::XV) * p.E + c) = make_uint4(0, 0, 0, 0);
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

template <typename T, int MODE>
cudaError_t by_states(const SsmParams &p, cudaStream_t s) {
    return p.S == 8 ? launch<T, 8, MODE>(p, s) : p.S == 16 ? launch<T, 16, MODE>(p, s)
                                            : p.S == 32 ? launch<T, 32, MODE>(p, s) : launch<T, 64, MODE>(p, s);
}

template <int MODE>
cudaError_t by_type(const SsmParams &p, la_dtype dt, cudaStream_t s) {
    return dt == LA_BF16 ? by_states<__nv_bfloat16, MODE>(p, s) : by_states<float, MODE>(p, s);
}

}  // namespace

int ssm_scan_channels(int S) { return kWarps * 32 / (S / spt_of(S)); }

cudaError_t ssm_scan(const SsmParams &p, la_dtype dt, cudaStream_t s) { return by_type<kScan>(p, dt, s); }

cudaError_t ssm_segments(const SsmParams &p, la_dtype dt, bool reverse, cudaStream_t s) {
    return reverse ? by_type<kReverse>(p, dt, s) : by_type<kSums>(p, dt, s);
}

}  // namespace la
