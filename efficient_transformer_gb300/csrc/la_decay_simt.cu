// la_decay_simt.cu -- decayed linear attention on the CUDA cores, float32 arithmetic: every
// dtype, width (32, 64, 128) and stride.
//
// Chunked pass: a block owns one segment of one key/value head and kSliceZ columns of z (out),
// and walks the segment in chunks of kChunk tokens with its DX x kSliceZ part of the state in
// shared memory:
//   P   = (X Y^T) o gamma^(i-j), j <= i          [C x C]
//   out = P Z + gamma^(i+1) X S                  [C x kSliceZ]
//   S   = gamma^C S + (gamma^(C-1-j) Y)^T Z      [DX x kSliceZ]
// The slices of one head repeat P (a third of the work at DX = 128) for two to four times the blocks.
#include "la_decay.cuh"

namespace la {
namespace {

constexpr int kChunk = 32, kSliceZ = kDecaySimtSlice, kThreads = 256;

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

// rows [t0, t0 + kChunk) (in the pass's order) x columns [c0, c0 + W) of a [N][*] matrix into smem
// rows of `ld` floats; rows past `valid` are zeros.
template <typename T, int W>
__device__ __forceinline__ void load_rows(float *dst, int ld, const T *src, long long stride, int n, int t0, int valid,
                                          int rev, int c0) {
    for (int idx = threadIdx.x; idx < kChunk * W; idx += kThreads) {
        const int r = idx / W, c = idx % W;
        const int t = rev ? n - 1 - (t0 + r) : t0 + r;
        dst[r * ld + c] = r < valid ? to_f32(src[t * stride + c0 + c]) : 0.f;
    }
}

// S (DX x kSliceZ, row stride kSliceZ) = gamma^valid S + sum_j gamma^(valid-1-j) y_j z_j^T; pw[n] = gamma^n.
template <int DX>
__device__ __forceinline__ void update_state(float *S, const float *Y, const float *Z, const float *pw, int valid,
                                             bool decay) {
    constexpr int R = DX / 16;   // state rows of a thread
    const int d0 = (threadIdx.x / 16) * R, e = (threadIdx.x % 16) * 2;
    float2 acc[R];
    const float g = decay ? pw[valid] : 1.f;
#pragma unroll
    for (int m = 0; m < R; ++m) {
        const float2 s = *reinterpret_cast<const float2 *>(&S[(d0 + m) * kSliceZ + e]);
        acc[m] = make_float2(s.x * g, s.y * g);
    }
    for (int j = 0; j < valid; ++j) {
        float2 z = *reinterpret_cast<const float2 *>(&Z[j * kSliceZ + e]);
        const float w = pw[valid - 1 - j];
        z.x *= w;
        z.y *= w;
#pragma unroll
        for (int m = 0; m < R; ++m) {
            const float y = Y[j * (DX + 4) + d0 + m];
            acc[m].x = fmaf(y, z.x, acc[m].x);
            acc[m].y = fmaf(y, z.y, acc[m].y);
        }
    }
#pragma unroll
    for (int m = 0; m < R; ++m) *reinterpret_cast<float2 *>(&S[(d0 + m) * kSliceZ + e]) = acc[m];
}

template <int DX>
constexpr int state_smem() {
    return (DX * kSliceZ + kChunk * (DX + 4) + kChunk * kSliceZ + kChunk + 4) * 4;
}

// The sum over one segment (see DecayStateParams); blockIdx.x = ((array, head), slice of Dv, segment).
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) k_decay_state(DecayStateParams p) {
    extern __shared__ float sm[];
    pdl_wait();
    float *S = sm, *Y = S + D * kSliceZ, *Z = Y + kChunk * (D + 4), *pw = Z + kChunk * kSliceZ;
    const int seg = blockIdx.x % (p.nseg - 1), rest = blockIdx.x / (p.nseg - 1);
    const int c0 = rest % (p.Dv / kSliceZ) * kSliceZ, ah = rest / (p.Dv / kSliceZ);
    const int a = ah / (p.B * p.Hkv), bg = ah % (p.B * p.Hkv), b = bg / p.Hkv, h = bg % p.Hkv;
    const float l2 = decay_log2(p.log_decay[h]);
    const Span sp = seg_span(decay_tokens(p.lengths, b, p.N), seg, p.seg_len);
    float *slots = p.slots[a] + (size_t)bg * p.nseg * p.D * p.Dv;
    if (seg == 0)
        for (int idx = threadIdx.x; idx < D * kSliceZ; idx += kThreads) {
            const size_t at = (size_t)(idx / kSliceZ) * p.Dv + c0 + idx % kSliceZ;
            slots[at] = p.init[a] ? p.init[a][(size_t)bg * p.D * p.Dv + at] * p.init_mul[a] : 0.f;
        }
    for (int idx = threadIdx.x; idx < D * kSliceZ; idx += kThreads) S[idx] = 0.f;
    if (threadIdx.x <= kChunk) pw[threadIdx.x] = exp2f(l2 * threadIdx.x);
    const int heads = p.heads[a], rev = p.rev[a];
    for (int t = sp.t0; t < sp.t1; t += kChunk) {
        const int valid = min(kChunk, sp.t1 - t);
        for (int r = 0; r < heads; ++r) {
            const long long hh = h * heads + r;
            __syncthreads();
            load_rows<T, D>(Y, D + 4, static_cast<const T *>(p.y[a]) + b * p.sy[a].b + hh * p.sy[a].h, p.sy[a].n, sp.n,
                            t, valid, rev, 0);
            load_rows<T, kSliceZ>(Z, kSliceZ, static_cast<const T *>(p.z[a]) + b * p.sz[a].b + hh * p.sz[a].h,
                                  p.sz[a].n, sp.n, t, valid, rev, c0);
            __syncthreads();
            update_state<D>(S, Y, Z, pw, valid, r == 0);
        }
    }
    __syncthreads();
    for (int idx = threadIdx.x; idx < D * kSliceZ; idx += kThreads)
        slots[(size_t)(seg + 1) * p.D * p.Dv + (size_t)(idx / kSliceZ) * p.Dv + c0 + idx % kSliceZ] = S[idx];
}

template <int DX>
constexpr int pass_smem() {
    return (DX * kSliceZ + 2 * kChunk * (DX + 4) + kChunk * kSliceZ + kChunk * (kChunk + 4) + kChunk + 4) * 4;
}

// A pass; blockIdx.x = (key/value head, slice of DZ, segment).
template <typename T, int DX>
__global__ void __launch_bounds__(kThreads) k_decay_pass(DecayParams p, int which) {
    extern __shared__ float sm[];
    pdl_wait();
    const DecayPass &ps = p.pass[which];
    float *S = sm, *X = S + DX * kSliceZ, *Y = X + kChunk * (DX + 4), *Z = Y + kChunk * (DX + 4);
    float *P = Z + kChunk * kSliceZ, *pw = P + kChunk * (kChunk + 4);
    const int DZ = ps.tr ? p.D : p.Dv;
    const int seg = blockIdx.x % p.nseg, rest = blockIdx.x / p.nseg, c0 = rest % (DZ / kSliceZ) * kSliceZ;
    const int bg = rest / (DZ / kSliceZ), b = bg / p.Hkv, h = bg % p.Hkv;
    const float l2 = decay_log2(p.log_decay[h]);
    const Span sp = seg_span(decay_tokens(p.lengths, b, p.N), seg, p.seg_len);
    const size_t E = (size_t)p.D * p.Dv;
    // the segment's starting state
    for (int idx = threadIdx.x; idx < DX * kSliceZ; idx += kThreads) {
        int d, e;   // consecutive threads take consecutive stored elements
        if (ps.tr) {
            d = idx % DX;
            e = idx / DX;
        } else {
            d = idx / kSliceZ;
            e = idx % kSliceZ;
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
        S[d * kSliceZ + e] = s;
    }
    if (threadIdx.x <= kChunk) pw[threadIdx.x] = exp2f(l2 * threadIdx.x);

    const int items = p.n_rep;
    const int i0 = threadIdx.x / 16, e0 = (threadIdx.x % 16) * 2, j0 = threadIdx.x % 16;
    float2 o[2];
    const T *xb = static_cast<const T *>(ps.x) + b * ps.sx.b, *yb = static_cast<const T *>(ps.y) + b * ps.sy.b,
            *zb = static_cast<const T *>(ps.z) + b * ps.sz.b;
    const int Hx = ps.many_yz ? p.Hkv : p.Hkv * p.n_rep;
    for (int t = sp.t0; t < sp.t1; t += kChunk) {
        const int valid = min(kChunk, sp.t1 - t);
        const int off = t == 0 ? ps.first_off : 0;
        for (int r = 0; r < items; ++r) {
            const long long hq = (long long)h * p.n_rep + r;
            const long long hx = ps.many_yz ? h : hq, hyz = ps.many_yz ? hq : h;
            __syncthreads();
            if (r == 0 || !ps.many_yz) load_rows<T, DX>(X, DX + 4, xb + hx * ps.sx.h, ps.sx.n, sp.n, t, valid, ps.rev, 0);
            if (r == 0 || ps.many_yz) {
                load_rows<T, DX>(Y, DX + 4, yb + hyz * ps.sy.h, ps.sy.n, sp.n, t, valid, ps.rev, 0);
                load_rows<T, kSliceZ>(Z, kSliceZ, zb + hyz * ps.sz.h, ps.sz.n, sp.n, t, valid, ps.rev, c0);
            }
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
            // out rows i0, i0 + 16 x columns e0, e0 + 1
            if (r == 0 || !ps.many_yz) {
                o[0] = o[1] = make_float2(0.f, 0.f);
                for (int d = 0; d < DX; d += 4) {
                    const float4 xa = *reinterpret_cast<const float4 *>(&X[i0 * (DX + 4) + d]);
                    const float4 xc = *reinterpret_cast<const float4 *>(&X[(i0 + 16) * (DX + 4) + d]);
                    const float *xav = &xa.x, *xcv = &xc.x;
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const float2 s = *reinterpret_cast<const float2 *>(&S[(d + q) * kSliceZ + e0]);
                        o[0].x = fmaf(xav[q], s.x, o[0].x);
                        o[0].y = fmaf(xav[q], s.y, o[0].y);
                        o[1].x = fmaf(xcv[q], s.x, o[1].x);
                        o[1].y = fmaf(xcv[q], s.y, o[1].y);
                    }
                }
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const float g = pw[i0 + 16 * q + 1 - off];
                    o[q].x *= g;
                    o[q].y *= g;
                }
            }
            for (int j = 0; j < valid; ++j) {
                const float2 z = *reinterpret_cast<const float2 *>(&Z[j * kSliceZ + e0]);
                const float pa = P[i0 * PL + j], pc = P[(i0 + 16) * PL + j];
                // z of a later token never meets an earlier row, not even as 0 z (z may be non-finite)
                if (j <= i0) {
                    o[0].x = fmaf(pa, z.x, o[0].x);
                    o[0].y = fmaf(pa, z.y, o[0].y);
                }
                if (j <= i0 + 16) {
                    o[1].x = fmaf(pc, z.x, o[1].x);
                    o[1].y = fmaf(pc, z.y, o[1].y);
                }
            }
            if (r == items - 1 || !ps.many_yz) {
                T *ob = static_cast<T *>(ps.out) + ((size_t)b * Hx + hx) * p.N * DZ + c0 + e0;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int i = i0 + 16 * q;
                    if (i < valid) {
                        const int tok = ps.rev ? sp.n - 1 - (t + i) : t + i;
                        ob[(size_t)tok * DZ] = from_f32<T>(p.scale * o[q].x);
                        ob[(size_t)tok * DZ + 1] = from_f32<T>(p.scale * o[q].y);
                    }
                }
            }
            // the state moves on once the chunk's last reader of the old one is done
            if (ps.many_yz) {
                __syncthreads();
                // S is read by r = 0 only; its decay, with the first power one lower where asked
                if (r == 0 && off) {
                    for (int idx = threadIdx.x; idx < DX * kSliceZ; idx += kThreads) S[idx] *= pw[valid - off];
                    __syncthreads();
                }
                update_state<DX>(S, Y, Z, pw, valid, r == 0 && !off);
            } else if (r == items - 1) {
                __syncthreads();
                if (off) {
                    for (int idx = threadIdx.x; idx < DX * kSliceZ; idx += kThreads) S[idx] *= pw[valid - off];
                    __syncthreads();
                }
                update_state<DX>(S, Y, Z, pw, valid, !off);
            }
        }
    }
    // rows past the sequence's length: zeros
    if (p.lengths) {
        const int z0 = max(sp.n, seg * p.seg_len), z1 = min(p.N, (seg + 1) * p.seg_len);
        for (int hh = 0; hh < (ps.many_yz ? 1 : p.n_rep); ++hh) {
            const long long hx = ps.many_yz ? h : (long long)h * p.n_rep + hh;
            T *ob = static_cast<T *>(ps.out) + ((size_t)b * Hx + hx) * p.N * DZ + c0;
            for (int idx = threadIdx.x; idx < (z1 - z0) * kSliceZ; idx += kThreads)
                ob[(size_t)(z0 + idx / kSliceZ) * DZ + idx % kSliceZ] = from_f32<T>(0.f);
        }
    }
    if (ps.fin && seg == p.nseg - 1) {
        __syncthreads();
        // what leaves a reverse pass decays once more; with no token at all it is what came in
        const float mul = ps.fin_mul * (ps.first_off ? exp2f(l2 * (sp.n > 0 ? ps.first_off : 0)) : 1.f);
        for (int idx = threadIdx.x; idx < DX * kSliceZ; idx += kThreads) {
            const int d = idx / kSliceZ, e = idx % kSliceZ;
            const size_t at = ps.tr ? (size_t)(c0 + e) * p.Dv + d : (size_t)d * p.Dv + c0 + e;
            ps.fin[(size_t)bg * E + at] = S[idx] * mul;
        }
    }
}

template <typename T, int D>
cudaError_t states_d(const DecayStateParams &p, cudaStream_t s) {
    auto kern = k_decay_state<T, D>;
    TraceScope tr("decay_state_simt", s);
    return launch_pdl(kern, dim3((p.nseg - 1) * (p.Dv / kSliceZ) * p.n * p.B * p.Hkv), dim3(kThreads), state_smem<D>(), s, p);
}

template <typename T, int DX>
cudaError_t pass_d(const DecayParams &p, int which, cudaStream_t s) {
    auto kern = k_decay_pass<T, DX>;
    constexpr int smem = pass_smem<DX>();
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return e;
    }
    const int DZ = p.pass[which].tr ? p.D : p.Dv;
    TraceScope tr("decay_pass_simt", s);
    return launch_pdl(kern, dim3(p.nseg * (DZ / kSliceZ) * p.B * p.Hkv), dim3(kThreads), smem, s, p, which);
}

template <typename T>
cudaError_t states_t(const DecayStateParams &p, cudaStream_t s) {
    return p.D == 32 ? states_d<T, 32>(p, s) : p.D == 64 ? states_d<T, 64>(p, s) : states_d<T, 128>(p, s);
}
template <typename T>
cudaError_t pass_t(const DecayParams &p, int which, cudaStream_t s) {
    const int DX = p.pass[which].tr ? p.Dv : p.D;
    return DX == 32 ? pass_d<T, 32>(p, which, s) : DX == 64 ? pass_d<T, 64>(p, which, s) : pass_d<T, 128>(p, which, s);
}

}  // namespace

cudaError_t decay_simt_states(const DecayStateParams &p, la_dtype dt, cudaStream_t s) {
    return dt == LA_BF16 ? states_t<__nv_bfloat16>(p, s) : states_t<float>(p, s);
}

cudaError_t decay_simt_pass(const DecayParams &p, int pass, la_dtype dt, cudaStream_t s) {
    return dt == LA_BF16 ? pass_t<__nv_bfloat16>(p, pass, s) : pass_t<float>(p, pass, s);
}

}  // namespace la
