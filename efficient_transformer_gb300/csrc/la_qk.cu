// la_qk.cu -- RMS norm of every query and key head with the position rotation, one pass over
// the data, forward and backward (la_qk_norm_rope_*).
//
//   y = Rot(x r w),  r = rsqrt(mean x^2 + eps)
//   u = Rot^T g,  dw = sum u x r,  dx = r (w u - x r mean(w u x r))
//
// Bound by memory: each row is read once and written once (the backward reads x and g).  A row of D
// elements lies in D / V neighbouring lanes, V = 16 bytes' worth each; such a group of lanes
// owns a token at a time and walks its heads, so that the token's cos and sin, with the weights in them
// (y[e] = r (x[e] w[e] c[e] + x[e'] w[e'] s[e]), e' the pair's other element), stay in registers; the
// partner's elements come by shuffles of the packed row.  kBatch heads' rows are loaded before the
// first is used, in the backward before the batch ahead of them is: its two sums a row are chains of
// shuffles that the loads run beside (2 x 32/8 heads, N 8192, D 128 bf16: 112 us without that, 95 us with it
// and a token's first rows loaded before its angles are found, 5.3 TB/s; 4 x 16/16 heads, N 4096, D 64: 51 and 44 us; in
// the forward the same costs registers, 222 -> 229 us).  The forward on 32/8 heads, N 65536, D 128:
// 222 us, 6.0 TB/s.
//
// Angles.  positions are 64-bit integers and inv_freq doubles, so an angle in float32, or even its
// reduction mod 2 pi there, would lose far positions.  inv_freq / 2 pi becomes a 64-bit binary fraction of a
// turn, rounded to nearest, and the integer product with the position wraps mod 2^64, i.e. mod one turn, exactly: the
// remaining error is |pos| 2^-65 turns (1.01 times that with inv_freq up to 1), before sincospif in float32, whose
// argument has 2^-26: so far positions are as good as near ones up to 2^39.
#include <cmath>

#include "la_internal.cuh"

namespace la {
namespace {

constexpr int kThreads = 256, kBatch = 4, kBatchBwd = 4;

struct QkParams {
    const void *x[2], *g[2];     // q and k rows; their output gradients (backward)
    Strides sx[2], sg[2];
    void *y[2];                  // outputs (forward: y, backward: dx), contiguous
    const void *w[2];            // weights or null
    int w_f32;
    int H[2], B, N;
    float eps;
    int normalize, rot, axes;
    int first_pair[5];           // pairs [first_pair[a], first_pair[a + 1]) belong to axis a
    const long long *pos;
    long long ps[3];
    const double *inv_freq;
    int heads_per_block;         // forward: heads of the joined list q, k that a block walks
    int y_blocks[2];             // backward: shares of q's and of k's heads (gridDim.y in all)
    float *part;                 // backward: [gridDim.y][gridDim.x][D] sums for the weights' gradients, or null
};

// inv_freq / 2 pi as a fraction of 2^64, wrapping: the double's 53-bit significand times
// round(2^66 / 2 pi) = 2^66 / 2 pi + 0.015, shifted to its place with one rounding (integer arithmetic: float64 units
// are few).
__device__ __forceinline__ unsigned long long turns_of(double f) {
    const unsigned long long bits = (unsigned long long)__double_as_longlong(f);
    const int e = (int)((bits >> 52) & 0x7ff);
    const unsigned long long m = (bits & 0xfffffffffffffull) | (e ? 1ull << 52 : 0ull);
    const unsigned long long k = 0xa2f9836e4e44152aull;
    const unsigned long long lo = m * k, hi = __umul64hi(m, k);
    const int sh = 54 - ((e ? e : 1) - 1023);   // m 2^(E - 52) / (2 pi) 2^64 = (m k) 2^(E - 54)
    unsigned long long r;
    if (sh >= 128)   // (the product has 117 bits)
        r = 0;
    else if (sh > 64)
        r = (hi >> (sh - 64)) + ((hi >> (sh - 65)) & 1);
    else if (sh == 64)
        r = hi + (lo >> 63);
    else if (sh > 0)
        r = ((hi << (64 - sh)) | (lo >> sh)) + ((lo >> (sh - 1)) & 1);
    else
        r = sh > -64 ? lo << -sh : 0;
    return (bits >> 63) ? 0ull - r : r;
}

template <typename T> struct Row;
template <> struct Row<float> {
    static constexpr int V = 4;
    static __device__ __forceinline__ void unpack(const uint4 &u, float *v) {
        v[0] = __uint_as_float(u.x);
        v[1] = __uint_as_float(u.y);
        v[2] = __uint_as_float(u.z);
        v[3] = __uint_as_float(u.w);
    }
    static __device__ __forceinline__ uint4 pack(const float *v) {
        return make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    }
};
template <> struct Row<__nv_bfloat16> {
    static constexpr int V = 8;
    static __device__ __forceinline__ void unpack(const uint4 &u, float *v) {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ uint4 pack(const float *v) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&h);
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
};

__device__ __forceinline__ unsigned long long pack2(float a, float b) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpack2(unsigned long long p) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(p));
    return r;
}
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

// A lane's 16 bytes of a row as V / 2 packed pairs of floats.
template <typename T>
__device__ __forceinline__ void unpack_row(const uint4 &u, unsigned long long *v) {
    float f[Row<T>::V];
    Row<T>::unpack(u, f);
#pragma unroll
    for (int i = 0; i < Row<T>::V / 2; ++i) v[i] = pack2(f[2 * i], f[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ uint4 pack_row(const unsigned long long *v) {
    float f[Row<T>::V];
#pragma unroll
    for (int i = 0; i < Row<T>::V / 2; ++i) {
        const float2 x = unpack2(v[i]);
        f[2 * i] = x.x;
        f[2 * i + 1] = x.y;
    }
    return Row<T>::pack(f);
}

// One lane's angles: the turned row is x[e] c[e] + partner[e] s[e].
template <typename T, int D, bool INTER>
struct Turn {
    static constexpr int V = Row<T>::V;                  // elements a lane
    static constexpr int PAIRS = V / 2;                  // pairs that it finds the angles of
    unsigned long long freq[PAIRS];                      // turns of them
    const long long *pos[PAIRS];                         // positions of their axes
    bool on, first;
    int src;                                             // lane of the partner's elements (split halves)

    __device__ __forceinline__ void init(const QkParams &p, int lane) {
        const int col = lane * V, half = p.rot / 2;
        on = col < p.rot;
        first = col < half;
        src = threadIdx.x % 32 + (INTER || !on ? 0 : first ? half / V : -(half / V));
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            // split halves: both lanes of a pair of lanes need all V angles, each finds half of them
            const int pair = INTER ? col / 2 + i : (first ? col : col - half + PAIRS) + i;
            int a = 0;
            while (on && a + 1 < p.axes && pair >= p.first_pair[a + 1]) ++a;
            pos[i] = p.pos + a * p.ps[0];
            freq[i] = on ? turns_of(p.inv_freq[pair]) : 0ull;
        }
    }
    // cos and sin of a token: c[e], s[e] (signed; the other way with `back`)
    __device__ __forceinline__ void at(const QkParams &p, int b, int n, bool back, float *c, float *s) const {
        float cs[PAIRS], sn[PAIRS];
        const long long off = b * p.ps[1] + n * p.ps[2];
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            const unsigned long long at = on ? (unsigned long long)pos[i][off] : 0ull;
            const int t = (int)((at * freq[i]) >> 32);   // turns in 2^-32, [-1/2, 1/2)
            sincospif((float)t * 4.656612873077393e-10f, &sn[i], &cs[i]);   // 2^-31: half turns
            if (back) sn[i] = -sn[i];
        }
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            if (INTER) {
                c[2 * i] = c[2 * i + 1] = cs[i];
                s[2 * i] = -sn[i];
                s[2 * i + 1] = sn[i];
            } else {
                const float co = __shfl_sync(0xffffffffu, cs[i], src), so = __shfl_sync(0xffffffffu, sn[i], src);
                c[i] = first ? cs[i] : co;
                c[PAIRS + i] = first ? co : cs[i];
                s[i] = first ? -sn[i] : so;
                s[PAIRS + i] = first ? -so : sn[i];
            }
        }
        if (!on) {
#pragma unroll
            for (int e = 0; e < V; ++e) {
                c[e] = 1.f;
                s[e] = 0.f;
            }
        }
    }
    // The partner's elements of a packed row; a lane that is not turned gets zeros (0 times whatever lies there).
    __device__ __forceinline__ uint4 partner(const uint4 &u) const {
        if (INTER) return u;
        uint4 r;
        r.x = __shfl_sync(0xffffffffu, u.x, src);
        r.y = __shfl_sync(0xffffffffu, u.y, src);
        r.z = __shfl_sync(0xffffffffu, u.z, src);
        r.w = __shfl_sync(0xffffffffu, u.w, src);
        return r;
    }
    // x c + partner s, packed pairs
    __device__ __forceinline__ void apply(const unsigned long long *x, const uint4 &raw, const unsigned long long *c,
                                          const unsigned long long *s, unsigned long long *y) const {
        unsigned long long o[V / 2];
        if (INTER) {
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                const float2 f = unpack2(x[i]);
                o[i] = pack2(f.y, f.x);
            }
        } else {
            unpack_row<T>(partner(raw), o);
        }
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            y[i] = mul2(x[i], c[i]);
            if (on) y[i] = fma2(o[i], s[i], y[i]);
        }
    }
};

template <int L>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int d = 1; d < L; d *= 2) x += __shfl_xor_sync(0xffffffffu, x, d);
    return x;
}

template <int V>
__device__ __forceinline__ void load_weights(const QkParams &p, int which, int col, float *w) {
#pragma unroll
    for (int e = 0; e < V; ++e)
        w[e] = !p.w[which] ? 1.f
               : p.w_f32   ? static_cast<const float *>(p.w[which])[col + e]
                           : __bfloat162float(static_cast<const __nv_bfloat16 *>(p.w[which])[col + e]);
}

// Blocks walk the tokens in strides of gridDim.x, kThreads / L at a time; blockIdx.y: heads_per_block heads.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 3) k_qk_fwd(QkParams p) {
    constexpr int V = Row<T>::V, L = D / V, kTok = kThreads / L;
    pdl_wait();
    const int lane = threadIdx.x % L;
    const unsigned ntok = (unsigned)p.B * p.N;   // below 2^31
    const int h0 = blockIdx.y * p.heads_per_block, h1 = min(h0 + p.heads_per_block, p.H[0] + p.H[1]);
    Turn<T, D, INTER> turn;
    turn.init(p, lane);
    for (unsigned t0 = blockIdx.x * kTok; t0 < ntok; t0 += gridDim.x * kTok) {
        const unsigned tok = t0 + threadIdx.x / L;
        const bool live = tok < ntok;
        const int b = live ? (int)(tok / (unsigned)p.N) : 0, n = live ? (int)(tok - (unsigned)b * p.N) : 0;
        float ct[V], st[V];
        turn.at(p, b, n, false, ct, st);
#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
            const int base = which ? p.H[0] : 0;
            const int lo = max(h0 - base, 0), hi = min(h1 - base, p.H[which]);
            if (lo >= hi) continue;
            unsigned long long c[V / 2], s[V / 2];
            {
                float w[V], wo[V];
                load_weights<V>(p, which, lane * V, w);
#pragma unroll
                for (int e = 0; e < V; ++e) wo[e] = INTER ? w[e ^ 1] : __shfl_sync(0xffffffffu, w[e], turn.src);
#pragma unroll
                for (int i = 0; i < V / 2; ++i) {
                    c[i] = pack2(ct[2 * i] * w[2 * i], ct[2 * i + 1] * w[2 * i + 1]);
                    s[i] = pack2(st[2 * i] * wo[2 * i], st[2 * i + 1] * wo[2 * i + 1]);
                }
            }
            const T *x = static_cast<const T *>(p.x[which]) + b * p.sx[which].b + n * p.sx[which].n + lane * V;
            T *y = static_cast<T *>(p.y[which]) + ((size_t)b * p.H[which] * p.N + n) * D + lane * V;
#pragma unroll 1
            for (int h = lo; h < hi; h += kBatch) {
                uint4 raw[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i)
                    raw[i] = live && h + i < hi ? *reinterpret_cast<const uint4 *>(x + (h + i) * p.sx[which].h)
                                                : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    unsigned long long v[V / 2], o[V / 2];
                    unpack_row<T>(raw[i], v);
                    turn.apply(v, raw[i], c, s, o);
                    if (p.normalize) {
                        unsigned long long q = 0ull;
#pragma unroll
                        for (int e = 0; e < V / 2; ++e) q = fma2(v[e], v[e], q);
                        const float2 ss = unpack2(q);
                        const float r = rsqrtf(row_sum<L>(ss.x + ss.y) * (1.f / D) + p.eps);
#pragma unroll
                        for (int e = 0; e < V / 2; ++e) o[e] = mul2(o[e], pack2(r, r));
                    }
                    if (live && h + i < hi) *reinterpret_cast<uint4 *>(y + (size_t)(h + i) * p.N * D) = pack_row<T>(o);
                }
            }
        }
    }
}

// Blocks walk the tokens in strides of gridDim.x and keep their part of a weight's gradient; blockIdx.y: a share
// of q's heads (the first y_blocks[0] of them) or of k's.
template <typename T, int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 2) k_qk_bwd(QkParams p) {
    constexpr int V = Row<T>::V, L = D / V, kTok = kThreads / L;
    __shared__ float red[kThreads / 32][D];
    pdl_wait();
    const int lane = threadIdx.x % L, which = (int)blockIdx.y >= p.y_blocks[0];
    const int h0 = (blockIdx.y - (which ? p.y_blocks[0] : 0)) * p.heads_per_block, h1 = min(h0 + p.heads_per_block, p.H[which]);
    const unsigned ntok = (unsigned)p.B * p.N;   // below 2^31
    unsigned long long dw[V / 2], w[V / 2];
    {
        float wf[V];
        load_weights<V>(p, which, lane * V, wf);
#pragma unroll
        for (int i = 0; i < V / 2; ++i) {
            w[i] = pack2(wf[2 * i], wf[2 * i + 1]);
            dw[i] = 0ull;
        }
    }
    Turn<T, D, INTER> turn;
    turn.init(p, lane);
    const Strides sx = which ? p.sx[1] : p.sx[0], sg = which ? p.sg[1] : p.sg[0];
    for (unsigned t0 = blockIdx.x * kTok; t0 < ntok; t0 += gridDim.x * kTok) {
        const unsigned tok = t0 + threadIdx.x / L;
        const bool live = tok < ntok;
        const int b = live ? (int)(tok / (unsigned)p.N) : 0, n = live ? (int)(tok - (unsigned)b * p.N) : 0;
        const T *x = static_cast<const T *>(which ? p.x[1] : p.x[0]) + b * sx.b + n * sx.n + lane * V;
        const T *g = static_cast<const T *>(which ? p.g[1] : p.g[0]) + b * sg.b + n * sg.n + lane * V;
        T *y = static_cast<T *>(which ? p.y[1] : p.y[0]) + ((size_t)b * p.H[which] * p.N + n) * D + lane * V;
        uint4 nx[kBatchBwd], ng[kBatchBwd];   // the next batch's rows
        auto fetch = [&](int h) {
#pragma unroll
            for (int i = 0; i < kBatchBwd; ++i) {
                const bool there = live && h + i < h1;
                ng[i] = there ? *reinterpret_cast<const uint4 *>(g + (h + i) * sg.h) : make_uint4(0u, 0u, 0u, 0u);
                nx[i] = there && p.normalize ? *reinterpret_cast<const uint4 *>(x + (h + i) * sx.h) : make_uint4(0u, 0u, 0u, 0u);
            }
        };
        fetch(h0);   // (the rows come while the angles are found)
        unsigned long long c[V / 2], s[V / 2];
        {
            float ct[V], st[V];
            turn.at(p, b, n, true, ct, st);
#pragma unroll
            for (int i = 0; i < V / 2; ++i) {
                c[i] = pack2(ct[2 * i], ct[2 * i + 1]);
                s[i] = pack2(st[2 * i], st[2 * i + 1]);
            }
        }
#pragma unroll 1
        for (int h = h0; h < h1; h += kBatchBwd) {
            uint4 rx[kBatchBwd], rg[kBatchBwd];
#pragma unroll
            for (int i = 0; i < kBatchBwd; ++i) {
                rx[i] = nx[i];
                rg[i] = ng[i];
            }
            if (h + kBatchBwd < h1) fetch(h + kBatchBwd);
#pragma unroll
            for (int i = 0; i < kBatchBwd; ++i) {
                const bool there = live && h + i < h1;
                unsigned long long u[V / 2], gv[V / 2];
                unpack_row<T>(rg[i], gv);
                turn.apply(gv, rg[i], c, s, u);
                if (p.normalize) {
                    unsigned long long v[V / 2], q = 0ull, m2 = 0ull;
                    unpack_row<T>(rx[i], v);
#pragma unroll
                    for (int e = 0; e < V / 2; ++e) q = fma2(v[e], v[e], q);
                    const float2 ss = unpack2(q);
                    // (rows that are not there are zeros and add nothing)
                    const float sum = row_sum<L>(ss.x + ss.y), r = there ? rsqrtf(sum * (1.f / D) + p.eps) : 0.f;
                    const unsigned long long r2 = pack2(r, r);
#pragma unroll
                    for (int e = 0; e < V / 2; ++e) {
                        v[e] = mul2(v[e], r2);                              // x r
                        dw[e] = fma2(u[e], v[e], dw[e]);
                        u[e] = mul2(u[e], w[e]);
                        m2 = fma2(u[e], v[e], m2);
                    }
                    const float2 mm = unpack2(m2);
                    const float m = row_sum<L>(mm.x + mm.y) * (-1.f / D);
                    const unsigned long long mneg = pack2(m, m);
#pragma unroll
                    for (int e = 0; e < V / 2; ++e) u[e] = mul2(r2, fma2(mneg, v[e], u[e]));
                }
                if (there) *reinterpret_cast<uint4 *>(y + (size_t)(h + i) * p.N * D) = pack_row<T>(u);
            }
        }
    }
    if (!p.part) return;
    // the block's sum: rows of the warp by shuffles, warps through shared memory
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float2 t2 = unpack2(dw[e / 2]);
        float t = e % 2 ? t2.y : t2.x;
#pragma unroll
        for (int d = L; d < 32; d *= 2) t += __shfl_xor_sync(0xffffffffu, t, d);
        if (threadIdx.x % 32 < L) red[threadIdx.x / 32][lane * V + e] = t;
    }
    __syncthreads();
    if (threadIdx.x < D) {
        float t = 0.f;
#pragma unroll
        for (int wp = 0; wp < kThreads / 32; ++wp) t += red[wp][threadIdx.x];
        p.part[((size_t)blockIdx.y * gridDim.x + blockIdx.x) * D + threadIdx.x] = t;
    }
}

// dw[which] = sum over the blocks' parts, in a fixed order; blockIdx.x = (which, 32 columns).
template <typename T>
__global__ void __launch_bounds__(1024) k_qk_dw(const float *part, int q_parts, int parts, int D, void *dq_w, void *dk_w,
                                                int w_f32) {
    __shared__ float red[32][33];
    pdl_wait();
    const int which = blockIdx.x / (D / 32), col = blockIdx.x % (D / 32) * 32 + threadIdx.x % 32, row = threadIdx.x / 32;
    float t = 0.f;
    for (int i = (which ? q_parts : 0) + row; i < (which ? parts : q_parts); i += 32) t += part[(size_t)i * D + col];
    red[row][threadIdx.x % 32] = t;
    __syncthreads();
    t = red[threadIdx.x % 32][row];   // a warp per column
#pragma unroll
    for (int d = 16; d > 0; d /= 2) t += __shfl_xor_sync(0xffffffffu, t, d);
    void *dst = which ? dk_w : dq_w;
    if (threadIdx.x % 32 == 0 && dst) {
        const int c = blockIdx.x % (D / 32) * 32 + row;
        if (w_f32)
            static_cast<float *>(dst)[c] = t;
        else
            static_cast<__nv_bfloat16 *>(dst)[c] = __float2bfloat16_rn(t);
    }
}

constexpr int kFwdBlocks = 6 * kPlanSms;   // blocks of the forward at most: two waves, each block with several tokens
constexpr int kBwdBlocks = 4 * kPlanSms;   // ... and of the backward (two an SM run at once)

// The backward's grid: heads in shares of at most 16, tokens over as many blocks as kBwdBlocks leaves.
struct BwdGrid {
    int heads, y[2], x;
};
BwdGrid bwd_grid(int B, int Hq, int Hkv, int N, int D, la_dtype dt) {
    BwdGrid g;
    g.heads = Hq < 16 ? Hq : 16;
    g.y[0] = (Hq + g.heads - 1) / g.heads;
    g.y[1] = (Hkv + g.heads - 1) / g.heads;
    const int tok = kThreads / (D / (dt == LA_BF16 ? 8 : 4));
    const long long groups = ((long long)B * N + tok - 1) / tok;
    const int most = kBwdBlocks / (g.y[0] + g.y[1]) > 1 ? kBwdBlocks / (g.y[0] + g.y[1]) : 1;
    g.x = groups < most ? (int)groups : most;
    return g;
}

template <typename T, int D, bool INTER>
cudaError_t fwd_launch(QkParams &p, cudaStream_t s) {
    constexpr int tok = kThreads / (D / Row<T>::V);
    const unsigned groups = (unsigned)(((long long)p.B * p.N + tok - 1) / tok);
    // few tokens: the heads are shared out, down to one batch a block, until every SM has two blocks
    const int H = p.H[0] + p.H[1];
    int hpb = H;
    while (hpb > kBatch && (long long)groups * ((H + hpb - 1) / hpb) < 2 * kPlanSms) hpb = (hpb + 1) / 2;
    p.heads_per_block = hpb;
    const unsigned blocks = groups < kFwdBlocks ? groups : kFwdBlocks;
    TraceScope tr("qk_norm_rope_fwd", s);
    return launch_pdl(k_qk_fwd<T, D, INTER>, dim3(blocks, (H + hpb - 1) / hpb), dim3(kThreads), 0, s, p);
}

template <typename T, int D, bool INTER>
cudaError_t bwd_launch(QkParams &p, void *dqw, void *dkw, cudaStream_t s) {
    const BwdGrid g = bwd_grid(p.B, p.H[0], p.H[1], p.N, D, sizeof(T) == 2 ? LA_BF16 : LA_F32);
    p.heads_per_block = g.heads;
    p.y_blocks[0] = g.y[0];
    p.y_blocks[1] = g.y[1];
    cudaError_t e;
    {
        TraceScope tr("qk_norm_rope_bwd", s);
        e = launch_pdl(k_qk_bwd<T, D, INTER>, dim3(g.x, g.y[0] + g.y[1]), dim3(kThreads), 0, s, p);
    }
    if (e != cudaSuccess || !p.part) return e;
    TraceScope tr("qk_norm_rope_dw", s);
    return launch_pdl(k_qk_dw<T>, dim3(2 * (D / 32)), dim3(1024), 0, s, static_cast<const float *>(p.part), g.x * g.y[0],
                      g.x * (g.y[0] + g.y[1]), D, dqw, dkw, p.w_f32);
}

template <typename T, int D>
cudaError_t launch_d(QkParams &p, bool bwd, bool inter, void *dqw, void *dkw, cudaStream_t s) {
    if (bwd) return inter ? bwd_launch<T, D, true>(p, dqw, dkw, s) : bwd_launch<T, D, false>(p, dqw, dkw, s);
    return inter ? fwd_launch<T, D, true>(p, s) : fwd_launch<T, D, false>(p, s);
}
template <typename T>
cudaError_t launch_t(QkParams &p, int D, bool bwd, bool inter, void *dqw, void *dkw, cudaStream_t s) {
    if (D == 32) return launch_d<T, 32>(p, bwd, inter, dqw, dkw, s);
    if (D == 64) return launch_d<T, 64>(p, bwd, inter, dqw, dkw, s);
    return launch_d<T, 128>(p, bwd, inter, dqw, dkw, s);
}

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

la_status check_sizes(int B, int Hq, int Hkv, int N, int D, int dtype) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || N <= 0 || D <= 0) return LA_ERR_ARG;
    if (dtype != LA_F32 && dtype != LA_BF16) return LA_ERR_ARG;
    if (((unsigned long long)B * N) >> 31 || Hq + (long long)Hkv >= 1 << 17) return LA_ERR_ARG;
    if (D != 32 && D != 64 && D != 128) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

// Strides of a [B, H, N, D] input; a dimension of one has no step.
la_status input_strides(const la_strides *st, int B, int H, int N, int D, int vec, Strides *out) {
    *out = contiguous_strides(H, N, D);
    if (!st) return LA_OK;
    if (st->b < 0 || st->h < 0 || st->n < 0) return LA_ERR_ARG;
    if (B > 1) out->b = st->b;
    if (H > 1) out->h = st->h;
    if (N > 1) out->n = st->n;
    return out->b % vec || out->h % vec || out->n % vec ? LA_ERR_ALIGN : LA_OK;
}

la_status run(bool bwd, const void *const *x, const void *const *g, void *const *y, void *dqw, void *dkw, int B, int Hq,
              int Hkv, int N, int D, la_dtype dt, const la_strides *const *sx, const la_strides *const *sg,
              const la_qk_args *a, void *ws, size_t ws_bytes, void *stream) {
    la_status st = check_sizes(B, Hq, Hkv, N, D, dt);
    if (st != LA_OK) return st;
    if (!a || !x[0] || !x[1] || !y[0] || !y[1] || (bwd && (!g[0] || !g[1]))) return LA_ERR_ARG;
    if (!(a->eps >= 0.f) || !std::isfinite(a->eps)) return LA_ERR_ARG;
    if (a->weight_dtype != LA_F32 && a->weight_dtype != dt) return LA_ERR_ARG;
    if (!a->normalize && (a->q_weight || a->k_weight || dqw || dkw)) return LA_ERR_ARG;
    if (a->rot < 0 || a->rot > D) return LA_ERR_ARG;
    if (a->rot % 16) return LA_ERR_UNSUPPORTED;
    QkParams p{};
    if (a->rot > 0) {
        if (!a->positions || !a->pos_strides || !a->inv_freq) return LA_ERR_ARG;
        if (a->axes < 1 || a->axes > 4 || (!a->sections && a->axes > 1)) return LA_ERR_ARG;
        long long pairs = 0;
        for (int i = 0; i < a->axes; ++i) {
            const int c = a->sections ? a->sections[i] : a->rot / 2;
            if (c < 0 || a->pos_strides[i < 3 ? i : 2] < 0) return LA_ERR_ARG;
            pairs += c;
            if (pairs > a->rot / 2) return LA_ERR_ARG;
            p.first_pair[i + 1] = (int)pairs;
        }
        if (pairs != a->rot / 2) return LA_ERR_ARG;
        for (int i = 0; i < 3; ++i) {
            if (a->pos_strides[i] < 0) return LA_ERR_ARG;
            p.ps[i] = a->pos_strides[i];
        }
        if (!aligned(a->positions, 8) || !aligned(a->inv_freq, 8)) return LA_ERR_ALIGN;
        p.axes = a->axes;
    }
    const void *ptrs[] = {x[0], x[1], bwd ? g[0] : nullptr, bwd ? g[1] : nullptr, y[0], y[1]};
    for (const void *q : ptrs)
        if (q && !aligned(q, 16)) return LA_ERR_ALIGN;
    const size_t wa = a->weight_dtype == LA_F32 ? 4 : 2;
    const void *wptrs[] = {a->q_weight, a->k_weight, dqw, dkw};
    for (const void *q : wptrs)
        if (q && !aligned(q, wa)) return LA_ERR_ALIGN;
    const int H[2] = {Hq, Hkv}, vec = dt == LA_BF16 ? 8 : 4;
    for (int i = 0; i < 2; ++i) {
        st = input_strides(sx[i], B, H[i], N, D, vec, &p.sx[i]);
        if (st == LA_OK && bwd) st = input_strides(sg[i], B, H[i], N, D, vec, &p.sg[i]);
        if (st != LA_OK) return st;
        p.x[i] = x[i];
        p.g[i] = bwd ? g[i] : nullptr;
        p.y[i] = y[i];
        p.H[i] = H[i];
    }
    if (bwd && (dqw || dkw)) {
        const size_t need = la_qk_norm_rope_workspace_size(B, Hq, Hkv, N, D, dt);
        if (!ws || ws_bytes < need) return LA_ERR_WORKSPACE;
        if (!aligned(ws, 256)) return LA_ERR_ALIGN;
        p.part = static_cast<float *>(ws);
    }
    p.w[0] = a->q_weight; p.w[1] = a->k_weight; p.w_f32 = a->weight_dtype == LA_F32;
    p.B = B; p.N = N; p.eps = a->eps; p.normalize = a->normalize ? 1 : 0; p.rot = a->rot;
    p.pos = a->positions; p.inv_freq = a->inv_freq;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool inter = a->interleaved != 0;
    cudaError_t e = dt == LA_BF16 ? launch_t<__nv_bfloat16>(p, D, bwd, inter, dqw, dkw, s)
                                  : launch_t<float>(p, D, bwd, inter, dqw, dkw, s);
    return e == cudaSuccess ? LA_OK : cuda_fail(e);
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

size_t la_qk_norm_rope_workspace_size(int B, int Hq, int Hkv, int N, int D, la_dtype dtype) {
    if (check_sizes(B, Hq, Hkv, N, D, dtype) != LA_OK) return 0;
    const BwdGrid g = bwd_grid(B, Hq, Hkv, N, D, dtype);
    return (size_t)g.x * (g.y[0] + g.y[1]) * D * sizeof(float);
}

la_status la_qk_norm_rope_fwd(const void *q, const void *k, void *q_out, void *k_out, int B, int Hq, int Hkv, int N,
                              int D, la_dtype dtype, const la_strides *q_strides, const la_strides *k_strides,
                              const la_qk_args *args, void *stream) {
    const void *x[2] = {q, k};
    void *y[2] = {q_out, k_out};
    const la_strides *sx[2] = {q_strides, k_strides};
    return run(false, x, nullptr, y, nullptr, nullptr, B, Hq, Hkv, N, D, dtype, sx, nullptr, args, nullptr, 0, stream);
}

la_status la_qk_norm_rope_bwd(const void *q, const void *k, const void *grad_q, const void *grad_k, void *dq, void *dk,
                              void *dq_weight, void *dk_weight, int B, int Hq, int Hkv, int N, int D, la_dtype dtype,
                              const la_strides *q_strides, const la_strides *k_strides, const la_strides *gq_strides,
                              const la_strides *gk_strides, const la_qk_args *args, void *workspace, size_t ws_bytes,
                              void *stream) {
    const void *x[2] = {q, k}, *g[2] = {grad_q, grad_k};
    void *y[2] = {dq, dk};
    const la_strides *sx[2] = {q_strides, k_strides}, *sg[2] = {gq_strides, gk_strides};
    return run(true, x, g, y, dq_weight, dk_weight, B, Hq, Hkv, N, D, dtype, sx, sg, args, workspace, ws_bytes, stream);
}

}  // extern "C"
