// la_decay_simt.cu -- decayed linear attention on the CUDA cores, float32 arithmetic: every
// dtype, width (32, 64, 128) and stride.
//
// Chunked pass: a block owns one segment of one key/value head and SZ columns of z (out),
// and walks the segment in chunks of kChunk tokens with its DX x SZ part of the state in
// shared memory:
//   P   = (X Y^T) o gamma^(i-j), j <= i          [C x C]
//   out = P Z + gamma^(i+1) X S                  [C x SZ]
//   S   = gamma^C S + (gamma^(C-1-j) Y)^T Z      [DX x SZ]
// SZ = 64 (32 where z is no wider): slices of one head repeat P, a third of the work at DX = 128; slices of 32 gave
// twice the blocks and were slower (gradients of 2 x 6/2 heads, N 777, D 64 float32: 68 us, with 64 columns 59).  Bound
// by the shared memory: 6 loads of 8 to 16 bytes for 16 FMA a thread with slices of 32, 76 % of its bandwidth where
// every SM had blocks, for 32 FMA with 64.  Two blocks an SM, as the registers hold the next chunk's rows.
#include "la_decay.cuh"

namespace la {
namespace {

constexpr int kChunk = 32, kThreads = 256;

// One segment's place: tokens [0, n) of the sequence along the pass's direction, this
// segment being [t0, t1) of them.
struct Span {
    int n, t0, t1;
};
__device__ __forceinline__ Span seg_span(int n, int seg, int seg_len) {
    Span s;
    s.n = n;
    s.t0 = min(n, seg * seg_len);
    s.t1 = min(n, s.t0 + seg_len);
    return s;
}

// Rows [t0, t0 + kChunk) (in the pass's order) x columns [c0, c0 + W) of a [N][*] matrix: fetched into registers
// while the chunk before is worked on, then put into smem rows of `ld` floats; rows past `valid` are zeros.
template <int W> struct Rows {
    static constexpr int K = kChunk * W / kThreads;
    float v[K];
    template <typename T>
    __device__ __forceinline__ void fetch(const T *src, long long stride, int n, int t0, int valid, int rev, int c0) {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int idx = threadIdx.x + i * kThreads, r = idx / W, c = idx % W;
            const int t = rev ? n - 1 - (t0 + r) : t0 + r;
            v[i] = r < valid ? to_f32(src[t * stride + c0 + c]) : 0.f;
        }
    }
    __device__ __forceinline__ void put(float *dst, int ld) const {
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int idx = threadIdx.x + i * kThreads;
            dst[(idx / W) * ld + idx % W] = v[i];
        }
    }
};

__device__ __forceinline__ void give2(float *dst, float a, float b) { *reinterpret_cast<float2 *>(dst) = make_float2(a, b); }
__device__ __forceinline__ void give2(__nv_bfloat16 *dst, float a, float b) {
    *reinterpret_cast<__nv_bfloat162 *>(dst) = __floats2bfloat162_rn(a, b);
}

// W floats from shared memory, 8 or 16 bytes at a time.
template <int W> __device__ __forceinline__ void take(float *r, const float *src) {
    if constexpr (W % 4 == 0) {
#pragma unroll
        for (int i = 0; i < W; i += 4) *reinterpret_cast<float4 *>(r + i) = *reinterpret_cast<const float4 *>(src + i);
    } else {
        *reinterpret_cast<float2 *>(r) = *reinterpret_cast<const float2 *>(src);
    }
}

// S (DX x SZ, row stride SZ) = gamma^valid S + sum_j gamma^(valid-1-j) y_j z_j^T; pw[n] = gamma^n.
template <int DX, int SZ>
__device__ __forceinline__ void update_state(float *S, const float *Y, const float *Z, const float *pw, int valid,
                                             bool decay) {
    constexpr int R = DX / 16, V = SZ / 16;   // state rows and columns of a thread
    const int d0 = (threadIdx.x / 16) * R, e = (threadIdx.x % 16) * V;
    float acc[R][V];
    const float g = decay ? pw[valid] : 1.f;
#pragma unroll
    for (int m = 0; m < R; ++m) {
        take<V>(acc[m], &S[(d0 + m) * SZ + e]);
#pragma unroll
        for (int c = 0; c < V; ++c) acc[m][c] *= g;
    }
    // in fours, so that the loads of the next tokens run beside the sums; rows past `valid` are zeros
    for (int j0 = 0; j0 < valid; j0 += 4) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int j = j0 + q;
            const float w = pw[max(valid - 1 - j, 0)];
            float y[R], z[V];
            take<R>(y, &Y[j * (DX + 4) + d0]);
            take<V>(z, &Z[j * SZ + e]);
#pragma unroll
            for (int c = 0; c < V; ++c) z[c] *= w;
#pragma unroll
            for (int m = 0; m < R; ++m)
#pragma unroll
                for (int c = 0; c < V; ++c) acc[m][c] = fmaf(y[m], z[c], acc[m][c]);
        }
    }
#pragma unroll
    for (int m = 0; m < R; ++m)
#pragma unroll
        for (int c = 0; c < V; c += 2)
            give2(&S[(d0 + m) * SZ + e + c], acc[m][c], acc[m][c + 1]);
}

template <int DX, int SZ>
constexpr int state_smem() {
    return (DX * SZ + kChunk * (DX + 4) + kChunk * SZ + kChunk + 4) * 4;
}

// The sum over one segment (see DecayStateParams); blockIdx.x = ((array, head), slice of Dv, segment).
template <typename T, int D, int SZ>
__global__ void __launch_bounds__(kThreads) k_decay_state(DecayStateParams p) {
    extern __shared__ float sm[];
    pdl_wait();
    float *S = sm, *Y = S + D * SZ, *Z = Y + kChunk * (D + 4), *pw = Z + kChunk * SZ;
    const int seg = blockIdx.x % (p.nseg - 1), rest = blockIdx.x / (p.nseg - 1);
    const int c0 = rest % (p.Dv / SZ) * SZ, ah = rest / (p.Dv / SZ);
    const int a = ah / (p.B * p.Hkv), bg = ah % (p.B * p.Hkv), b = bg / p.Hkv, h = bg % p.Hkv;
    const float l2 = decay_log2(p.log_decay[h]);
    const Span sp = seg_span(decay_tokens(p.lengths, b, p.N), seg, p.seg_len);
    float *slots = p.slots[a] + (size_t)bg * p.nseg * p.D * p.Dv;
    if (seg == 0)
        for (int idx = threadIdx.x; idx < D * SZ; idx += kThreads) {
            const size_t at = (size_t)(idx / SZ) * p.Dv + c0 + idx % SZ;
            slots[at] = p.init[a] ? p.init[a][(size_t)bg * p.D * p.Dv + at] * p.init_mul[a] : 0.f;
        }
    for (int idx = threadIdx.x; idx < D * SZ; idx += kThreads) S[idx] = 0.f;
    if (threadIdx.x <= kChunk) pw[threadIdx.x] = exp2f(l2 * threadIdx.x);
    const int heads = p.heads[a], rev = p.rev[a];
    Rows<D> ry;
    Rows<SZ> rz;
    auto fetch = [&](int t, int r) {
        const long long hh = h * heads + r;
        const int valid = min(kChunk, sp.t1 - t);
        ry.fetch(static_cast<const T *>(p.y[a]) + b * p.sy[a].b + hh * p.sy[a].h, p.sy[a].n, sp.n, t, valid, rev, 0);
        rz.fetch(static_cast<const T *>(p.z[a]) + b * p.sz[a].b + hh * p.sz[a].h, p.sz[a].n, sp.n, t, valid, rev, c0);
    };
    if (sp.t0 < sp.t1) fetch(sp.t0, 0);
    for (int t = sp.t0; t < sp.t1; t += kChunk) {
        const int valid = min(kChunk, sp.t1 - t);
        for (int r = 0; r < heads; ++r) {
            __syncthreads();
            ry.put(Y, D + 4);
            rz.put(Z, SZ);
            if (r + 1 < heads)
                fetch(t, r + 1);
            else if (t + kChunk < sp.t1)
                fetch(t + kChunk, 0);
            __syncthreads();
            update_state<D, SZ>(S, Y, Z, pw, valid, r == 0);
        }
    }
    __syncthreads();
    for (int idx = threadIdx.x; idx < D * SZ; idx += kThreads)
        slots[(size_t)(seg + 1) * p.D * p.Dv + (size_t)(idx / SZ) * p.Dv + c0 + idx % SZ] = S[idx];
}

template <int DX, int SZ>
constexpr int pass_smem() {
    return (DX * SZ + 2 * kChunk * (DX + 4) + kChunk * SZ + kChunk * (kChunk + 4) + kChunk + 4) * 4;
}

// npass passes; blockIdx.x = (key/value head, slice of DZ, segment, pass).
template <typename T, int DX, int SZ>
__global__ void __launch_bounds__(kThreads, 2) k_decay_pass(const __grid_constant__ DecayParams p, int pass0, int npass) {
    extern __shared__ float sm[];
    pdl_wait();
    const DecayPass &ps = p.pass[pass0 + blockIdx.x % npass];
    float *S = sm, *X = S + DX * SZ, *Y = X + kChunk * (DX + 4), *Z = Y + kChunk * (DX + 4);
    float *P = Z + kChunk * SZ, *pw = P + kChunk * (kChunk + 4);
    const int DZ = ps.tr ? p.D : p.Dv;
    const int bx = blockIdx.x / npass, seg = bx % p.nseg, rest = bx / p.nseg, c0 = rest % (DZ / SZ) * SZ;
    const int bg = rest / (DZ / SZ), b = bg / p.Hkv, h = bg % p.Hkv;
    const float l2 = decay_log2(p.log_decay[h]);
    const Span sp = seg_span(decay_tokens(p.lengths, b, p.N), seg, p.seg_len);
    const size_t E = (size_t)p.D * p.Dv;
    // the segment's starting state
    for (int idx = threadIdx.x; idx < DX * SZ; idx += kThreads) {
        int d, e;   // consecutive threads take consecutive stored elements
        if (ps.tr) {
            d = idx % DX;
            e = idx / DX;
        } else {
            d = idx / SZ;
            e = idx % SZ;
        }
        const size_t at = ps.tr ? (size_t)(c0 + e) * p.Dv + d : (size_t)d * p.Dv + c0 + e;
        float s = 0.f;
        if (p.nseg == 1) {
            if (ps.init) s = ps.init[(size_t)bg * E + at] * ps.init_mul;
        } else {
            const float *sl = ps.slots + (size_t)bg * p.nseg * E + at;
            s = sl[0] * (seg > 0 ? exp2f(l2 * (sp.t0 - ps.first_off)) : 1.f);
            for (int u = 1; u <= seg; ++u) {
                const int end = min(sp.n, u * p.seg_len);   // tokens up to the end of segment u - 1
                s = fmaf(exp2f(l2 * (sp.t0 - end)), sl[(size_t)u * E], s);
            }
        }
        S[d * SZ + e] = s;
    }
    if (threadIdx.x <= kChunk) pw[threadIdx.x] = exp2f(l2 * threadIdx.x);

    const int items = p.n_rep;
    constexpr int V = SZ / 16;   // output columns of a thread
    const int i0 = threadIdx.x / 16, e0 = (threadIdx.x % 16) * V, j0 = threadIdx.x % 16;
    float o[2][V];
    const T *xb = static_cast<const T *>(ps.x) + b * ps.sx.b, *yb = static_cast<const T *>(ps.y) + b * ps.sy.b,
            *zb = static_cast<const T *>(ps.z) + b * ps.sz.b;
    const int Hx = ps.many_yz ? p.Hkv : p.Hkv * p.n_rep;
    Rows<DX> rx, ry;
    Rows<SZ> rz;
    auto fetch = [&](int t, int r) {
        const long long hq = (long long)h * p.n_rep + r, hx = ps.many_yz ? h : hq, hyz = ps.many_yz ? hq : h;
        const int valid = min(kChunk, sp.t1 - t);
        if (r == 0 || !ps.many_yz) rx.fetch(xb + hx * ps.sx.h, ps.sx.n, sp.n, t, valid, ps.rev, 0);
        if (r == 0 || ps.many_yz) {
            ry.fetch(yb + hyz * ps.sy.h, ps.sy.n, sp.n, t, valid, ps.rev, 0);
            rz.fetch(zb + hyz * ps.sz.h, ps.sz.n, sp.n, t, valid, ps.rev, c0);
        }
    };
    if (sp.t0 < sp.t1) fetch(sp.t0, 0);
    for (int t = sp.t0; t < sp.t1; t += kChunk) {
        const int valid = min(kChunk, sp.t1 - t);
        const int off = t == 0 ? ps.first_off : 0;
        for (int r = 0; r < items; ++r) {
            const long long hx = ps.many_yz ? h : (long long)h * p.n_rep + r;
            __syncthreads();
            if (r == 0 || !ps.many_yz) rx.put(X, DX + 4);
            if (r == 0 || ps.many_yz) {
                ry.put(Y, DX + 4);
                rz.put(Z, SZ);
            }
            if (r + 1 < items)
                fetch(t, r + 1);
            else if (t + kChunk < sp.t1)
                fetch(t + kChunk, 0);
            __syncthreads();
            // P, rows i0, i0 + 16 x columns j0, j0 + 16
            float s00 = 0.f, s01 = 0.f, s10 = 0.f, s11 = 0.f;
            for (int d = 0; d < DX; d += 4) {
                const float4 xa = *reinterpret_cast<const float4 *>(&X[i0 * (DX + 4) + d]);
                const float4 xc = *reinterpret_cast<const float4 *>(&X[(i0 + 16) * (DX + 4) + d]);
                const float4 ya = *reinterpret_cast<const float4 *>(&Y[j0 * (DX + 4) + d]);
                const float4 yc = *reinterpret_cast<const float4 *>(&Y[(j0 + 16) * (DX + 4) + d]);
                s00 = fmaf(xa.x, ya.x, fmaf(xa.y, ya.y, fmaf(xa.z, ya.z, fmaf(xa.w, ya.w, s00))));
                s01 = fmaf(xa.x, yc.x, fmaf(xa.y, yc.y, fmaf(xa.z, yc.z, fmaf(xa.w, yc.w, s01))));
                s10 = fmaf(xc.x, ya.x, fmaf(xc.y, ya.y, fmaf(xc.z, ya.z, fmaf(xc.w, ya.w, s10))));
                s11 = fmaf(xc.x, yc.x, fmaf(xc.y, yc.y, fmaf(xc.z, yc.z, fmaf(xc.w, yc.w, s11))));
            }
            constexpr int PL = kChunk + 4;
            P[i0 * PL + j0] = j0 <= i0 ? s00 * pw[i0 - j0] : 0.f;
            P[i0 * PL + j0 + 16] = 0.f;   // j0 + 16 > i0
            P[(i0 + 16) * PL + j0] = s10 * pw[i0 + 16 - j0];
            P[(i0 + 16) * PL + j0 + 16] = j0 <= i0 ? s11 * pw[i0 - j0] : 0.f;
            (void)s01;
            __syncthreads();
            // out rows i0, i0 + 16 x columns e0 .. e0 + V
            if (r == 0 || !ps.many_yz) {
#pragma unroll
                for (int c = 0; c < V; ++c) o[0][c] = o[1][c] = 0.f;
                for (int d = 0; d < DX; d += 4) {
                    float xa[4], xc[4], sv[V];
                    take<4>(xa, &X[i0 * (DX + 4) + d]);
                    take<4>(xc, &X[(i0 + 16) * (DX + 4) + d]);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        take<V>(sv, &S[(d + q) * SZ + e0]);
#pragma unroll
                        for (int c = 0; c < V; ++c) {
                            o[0][c] = fmaf(xa[q], sv[c], o[0][c]);
                            o[1][c] = fmaf(xc[q], sv[c], o[1][c]);
                        }
                    }
                }
                const float ga = pw[i0 + 1 - off], gc = pw[i0 + 17 - off];
#pragma unroll
                for (int c = 0; c < V; ++c) {
                    o[0][c] *= ga;
                    o[1][c] *= gc;
                }
            }
            for (int jb = 0; jb < valid; jb += 4) {
                float pa[4], pc[4], z[V];
                take<4>(pa, &P[i0 * PL + jb]);
                take<4>(pc, &P[(i0 + 16) * PL + jb]);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int j = jb + q;
                    take<V>(z, &Z[j * SZ + e0]);
                    // z of a later token never meets an earlier row, not even as 0 z (z may be non-finite)
                    if (j <= i0) {
#pragma unroll
                        for (int c = 0; c < V; ++c) o[0][c] = fmaf(pa[q], z[c], o[0][c]);
                    }
                    if (j <= i0 + 16) {
#pragma unroll
                        for (int c = 0; c < V; ++c) o[1][c] = fmaf(pc[q], z[c], o[1][c]);
                    }
                }
            }
            if (r == items - 1 || !ps.many_yz) {
                T *ob = static_cast<T *>(ps.out) + ((size_t)b * Hx + hx) * p.N * DZ + c0 + e0;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int i = i0 + 16 * q;
                    if (i < valid) {
                        const int tok = ps.rev ? sp.n - 1 - (t + i) : t + i;
#pragma unroll
                        for (int c = 0; c < V; c += 2)
                            give2(ob + (size_t)tok * DZ + c, p.scale * o[q][c], p.scale * o[q][c + 1]);
                    }
                }
            }
            // the state moves on once the chunk's last reader of the old one is done
            if (ps.many_yz) {
                __syncthreads();
                // S is read by r = 0 only; its decay, with the first power one lower where asked
                if (r == 0 && off) {
                    for (int idx = threadIdx.x; idx < DX * SZ; idx += kThreads) S[idx] *= pw[valid - off];
                    __syncthreads();
                }
                update_state<DX, SZ>(S, Y, Z, pw, valid, r == 0 && !off);
            } else if (r == items - 1) {
                __syncthreads();
                if (off) {
                    for (int idx = threadIdx.x; idx < DX * SZ; idx += kThreads) S[idx] *= pw[valid - off];
                    __syncthreads();
                }
                update_state<DX, SZ>(S, Y, Z, pw, valid, !off);
            }
        }
    }
    // rows past the sequence's length: zeros
    if (p.lengths) {
        const int z0 = max(sp.n, seg * p.seg_len), z1 = min(p.N, (seg + 1) * p.seg_len);
        for (int hh = 0; hh < (ps.many_yz ? 1 : p.n_rep); ++hh) {
            const long long hx = ps.many_yz ? h : (long long)h * p.n_rep + hh;
            T *ob = static_cast<T *>(ps.out) + ((size_t)b * Hx + hx) * p.N * DZ + c0;
            for (int idx = threadIdx.x; idx < (z1 - z0) * SZ; idx += kThreads)
                ob[(size_t)(z0 + idx / SZ) * DZ + idx % SZ] = from_f32<T>(0.f);
        }
    }
    if (ps.fin && seg == p.nseg - 1) {
        __syncthreads();
        // what leaves a reverse pass decays once more; with no token at all it is what came in
        const float mul = ps.fin_mul * (ps.first_off ? exp2f(l2 * (sp.n > 0 ? ps.first_off : 0)) : 1.f);
        for (int idx = threadIdx.x; idx < DX * SZ; idx += kThreads) {
            const int d = idx / SZ, e = idx % SZ;
            const size_t at = ps.tr ? (size_t)(c0 + e) * p.Dv + d : (size_t)d * p.Dv + c0 + e;
            ps.fin[(size_t)bg * E + at] = S[idx] * mul;
        }
    }
}

template <typename K> cudaError_t allow_smem(K kern, int smem) {
    return smem > 48 * 1024 ? cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) : cudaSuccess;
}

template <typename T, int D, int SZ> cudaError_t states_of(const DecayStateParams &p, cudaStream_t s) {
    auto kern = k_decay_state<T, D, SZ>;
    constexpr int smem = state_smem<D, SZ>();
    cudaError_t e = allow_smem(kern, smem);
    if (e != cudaSuccess) return e;
    TraceScope tr("decay_state_simt", s);
    return launch_pdl(kern, dim3((p.nseg - 1) * (p.Dv / SZ) * p.n * p.B * p.Hkv), dim3(kThreads), smem, s, p);
}

template <typename T, int DX, int SZ>
cudaError_t passes_of(const DecayParams &p, int pass0, int npass, int DZ, cudaStream_t s) {
    auto kern = k_decay_pass<T, DX, SZ>;
    constexpr int smem = pass_smem<DX, SZ>();
    cudaError_t e = allow_smem(kern, smem);
    if (e != cudaSuccess) return e;
    TraceScope tr("decay_pass_simt", s);
    return launch_pdl(kern, dim3((unsigned)npass * p.nseg * (DZ / SZ) * p.B * p.Hkv), dim3(kThreads), smem, s, p, pass0,
                      npass);
}

template <typename T, int SZ> cudaError_t states_sz(const DecayStateParams &p, cudaStream_t s) {
    return p.D == 32   ? states_of<T, 32, SZ>(p, s)
           : p.D == 64 ? states_of<T, 64, SZ>(p, s)
                       : states_of<T, 128, SZ>(p, s);
}
template <typename T> cudaError_t states_t(const DecayStateParams &p, cudaStream_t s) {
    return decay_simt_slice(p.Dv) == 32 ? states_sz<T, 32>(p, s) : states_sz<T, 64>(p, s);
}

template <typename T, int SZ>
cudaError_t passes_sz(const DecayParams &p, int pass0, int npass, int DX, int DZ, cudaStream_t s) {
    return DX == 32   ? passes_of<T, 32, SZ>(p, pass0, npass, DZ, s)
           : DX == 64 ? passes_of<T, 64, SZ>(p, pass0, npass, DZ, s)
                      : passes_of<T, 128, SZ>(p, pass0, npass, DZ, s);
}
template <typename T> cudaError_t passes_t(const DecayParams &p, int pass0, int npass, cudaStream_t s) {
    const int tr = p.pass[pass0].tr, DX = tr ? p.Dv : p.D, DZ = tr ? p.D : p.Dv;
    return decay_simt_slice(DZ) == 32 ? passes_sz<T, 32>(p, pass0, npass, DX, DZ, s)
                                      : passes_sz<T, 64>(p, pass0, npass, DX, DZ, s);
}

}  // namespace

cudaError_t decay_simt_states(const DecayStateParams &p, la_dtype dt, cudaStream_t s) {
    return dt == LA_BF16 ? states_t<__nv_bfloat16>(p, s) : states_t<float>(p, s);
}

cudaError_t decay_simt_passes(const DecayParams &p, int pass0, int npass, la_dtype dt, cudaStream_t s) {
    return dt == LA_BF16 ? passes_t<__nv_bfloat16>(p, pass0, npass, s) : passes_t<float>(p, pass0, npass, s);
}

}  // namespace la
