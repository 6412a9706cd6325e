// la_decay_tc.cu -- decayed linear attention on the tensor cores (tcgen05 / TMEM / TMA), bfloat16.
//
// One block walks one segment of one key/value head in chunks of C = 128 tokens.  Per chunk (X, Y, Z:
// see la_decay.cuh; W_ij = gamma^(i-j) for j <= i, else 0):
//   A   = X Y^T                                  [C x C]     scores
//   P   = bf16(A o W), in TMEM                               (fp32 decay, one rounding)
//   O   = X S_bf, then row i times gamma^(i+1), in TMEM
//   O  += P Z                                    [C x DZ]
//   S   = gamma^C S + (gamma^(C-1-j) y_j)^T Z    [DX x DZ]   fp32 in TMEM
// Powers of gamma are only ever of whole distances >= 0, so no decay overflows.  The decayed Y^T is an
// operand made from Y: it is split into two bf16 terms (hi + lo, 2^-17 relative) and both are multiplied,
// because what it sums is a float32 output (the state); one rounding would leave 2^-9 there.
// P and S_bf are rounded once: they only reach bf16 outputs.
//
// Operands made by the CUDA cores go to TMEM (P over the scores it comes from, Y^T hi and lo), which
// leaves the shared memory to two stages of every TMA tile.  TMEM columns: S, O, scores / P, Y^T hi | lo.
// Several heads of x share one chunk of y, z (grouped queries; S moves on after the last), or several heads
// of y, z share one of x (their gradients; O and S sum over the heads).
//
// Warps: 0 TMA, 1 MMA of scores and P Z, 2 MMA of X S_bf and the state, 4-7 P, 8-11 S -> S_bf and the decay of S, 12-15 O's row powers and the output,
// 16-23 Y^T (and the zeros past a sequence's length).
//
// The reverse passes (gradients of k and v) take the same steps with j >= i and gamma^(j-i), chunks from the
// last to the first.
#include "la_decay.cuh"
#include "la_tc_common.cuh"

namespace la {
namespace {

constexpr int C = kDecayTcChunk;
constexpr int kMainThreads = 768, kYtThreads = 256;

struct PassMaps {
    CUtensorMap m[3][4];   // per pass: x, y, z, out
};

template <int DX, int DZ>
struct MainCfg {
    static constexpr int X_BYTES = C * (DX > DZ ? DX : DZ) * 2;   // also stages the output tile
    static constexpr int Y_BYTES = C * DX * 2, Z_BYTES = C * DZ * 2, YZ_BYTES = Y_BYTES + Z_BYTES;
    static constexpr int S_BYTES = DX * DZ * 2;
    static constexpr int BUDGET = kSmemLimit - 1024 - 2048;   // alignment; barriers and tables
    static constexpr int NX = (BUDGET - S_BYTES) / (2 * (X_BYTES + YZ_BYTES)) >= 2 ? 4 : 2;
    static constexpr int NY_FIT = (BUDGET - S_BYTES - NX * X_BYTES) / YZ_BYTES;
    static constexpr int NY = NY_FIT > 4 ? 4 : NY_FIT;
    static constexpr int SMEM = NX * X_BYTES + NY * YZ_BYTES + S_BYTES + 1024;
    static_assert(NY >= 2, "two stages");
    static constexpr int T_S = 0, T_O = 128, T_A = 256, T_YH = 384, T_YL = 448;
};

// A block's part of the sequence: tokens [lo, hi), `before` tokens of the sequence precede it in the pass's
// order.
struct Part {
    int lo, hi, before;
};
__device__ __forceinline__ Part part_of(int n, int N, int u, int nseg, int seg_len, int rev) {
    const int s = rev ? nseg - 1 - u : u;
    Part r;
    r.lo = min(n, s * seg_len);
    r.hi = min(n, r.lo + seg_len);
    r.before = rev ? n - r.hi : r.lo;
    return r;
}

// a b for two pairs of floats (one packed instruction).
__device__ __forceinline__ void mul2(float &x, float &y, float a, float b) {
    unsigned long long p, q;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(q) : "f"(a), "f"(b));
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(p) : "l"(q));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
}

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t u) { return *reinterpret_cast<__nv_bfloat162 *>(&u); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 h) { return *reinterpret_cast<uint32_t *>(&h); }

// The decays w of 64 tokens (8 groups of 8) of which a thread meets 2 in each group, as two bf16 terms.
struct YtWeights {
    uint32_t hi[8], lo[8];
    __device__ __forceinline__ void set(const float *w, float mul) {
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            const float a = w[8 * g + 2 * (threadIdx.x % 4)] * mul, b = w[8 * g + 2 * (threadIdx.x % 4) + 1] * mul;
            hi[g] = pack_bf16x2(a, b);
            const float2 f = unpack_bf16x2(hi[g]);
            lo[g] = pack_bf16x2(a - f.x, b - f.y);
        }
    }
};

// Decayed Y^T of one tile for the warp's 32 lanes d and the 64 tokens from j0: y w as two bf16 terms, into
// 32 columns each at th and tl.  With w = wh + wl (bf16 each), hi = bf16(y wh), the remainder y wh - hi is exact in
// bf16 (one fused multiply-add) and lo = bf16(remainder + y wl): three packed operations a pair, 2^-17 relative in
// all.  The tile's 8 x 8 blocks come transposed out of shared memory in the layout of the store.
// Tokens at or past `valid` count as zeros whatever they hold.
__device__ __forceinline__ void yt_block(const uint8_t *y, int d0, int j0, const YtWeights &w, int valid, uint32_t th,
                                         uint32_t tl) {
    const int t = threadIdx.x % 32;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {   // lanes d0 + 16 half ..
        const uint32_t addr = smem_u32(y) + swz_chunk(C, j0 + 8 * (t / 16) + t % 8, (d0 + 16 * half) / 8 + ((t / 8) & 1));
        uint32_t v[16], hi[16], lo[16];
#pragma unroll
        for (int q = 0; q < 4; ++q) ldmatrix_x4_trans(addr + q * 16 * 128, v + 4 * q);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int g = i / 2;   // group of 8 tokens
            uint32_t u = v[i];
            if (valid < C) {
                const int j = j0 + 8 * g + 2 * (t % 4);
                u = j + 1 < valid ? u : j < valid ? u & 0xffffu : 0u;
            }
            const __nv_bfloat162 wh = as_bf162(w.hi[g]), h = __hmul2(as_bf162(u), wh);
            const __nv_bfloat162 r = __hfma2(as_bf162(u), wh, __hneg2(h));
            hi[i] = as_u32(h);
            lo[i] = as_u32(__hfma2(as_bf162(u), as_bf162(w.lo[g]), r));
        }
        tmem_st_frag32(th + ((uint32_t)(16 * half) << 16), hi);
        tmem_st_frag32(tl + ((uint32_t)(16 * half) << 16), lo);
    }
}

// Zero rows [valid, C) of a C x W tile (what lies past a sequence's length must not meet the MMA, where 0
// times a non-finite value is not 0); nth threads, this one being i.
template <int W>
__device__ __forceinline__ void zero_rows(uint8_t *tile, int valid, int i, int nth) {
    for (int idx = i; idx < (C - valid) * (W / 8); idx += nth)
        *reinterpret_cast<uint4 *>(tile + swz_chunk(C, valid + idx / (W / 8), idx % (W / 8))) = make_uint4(0u, 0u, 0u, 0u);
}

template <int DX, int DZ>
__global__ void __launch_bounds__(kMainThreads, 1) k_decay_tc(const __grid_constant__ PassMaps maps,
                                                              const __grid_constant__ DecayParams p, int pass0,
                                                              int npass) {
    using K = MainCfg<DX, DZ>;
    constexpr int NX = K::NX, NY = K::NY;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t x_full[NX], x_empty[NX], yz_full[NY], yz_empty[NY];
    __shared__ uint64_t sc_full, p_ready, o_inter, o_scaled, o_full, o_free, s_full, s_conv, yt_ready, yt_done, fin[2];
    __shared__ __align__(16) float pw[C + 4], wtab[2][C];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    uint8_t *xbuf = align1024(smem_raw);
    uint8_t *yzbuf = xbuf + NX * K::X_BYTES;
    uint8_t *sbf = yzbuf + NY * K::YZ_BYTES;

    pdl_wait();
    const int warp = threadIdx.x / 32;
    const int pi = pass0 + blockIdx.x % npass, rest = blockIdx.x / npass;
    const DecayPass &ps = p.pass[pi];
    const CUtensorMap *mx = &maps.m[pi][0], *my = &maps.m[pi][1], *mz = &maps.m[pi][2], *mo = &maps.m[pi][3];
    const int u = rest % p.nseg, bg = rest / p.nseg, b = bg / p.Hkv, h = bg % p.Hkv;
    const int n = decay_tokens(p.lengths, b, p.N), rev = ps.rev, many = ps.many_yz, reps = p.n_rep;
    const Part part = part_of(n, p.N, u, p.nseg, p.seg_len, rev);
    const int nchunk = (part.hi - part.lo + C - 1) / C;
    const int off0 = u == 0 ? ps.first_off : 0;   // of the first chunk
    const float l2 = decay_log2(p.log_decay[h]);
    auto chunk0 = [&](int k) { return part.lo + C * (rev ? nchunk - 1 - k : k); };
    // tokens of the short chunk (the last in token order)
    const int vlast = part.hi - part.lo - C * (nchunk - 1);

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < NX; ++s) {
            mbar_init(&x_full[s], 1);
            mbar_init(&x_empty[s], 4);
        }
        for (int s = 0; s < NY; ++s) {
            mbar_init(&yz_full[s], 1);
            mbar_init(&yz_empty[s], 2);
        }
        mbar_init(&sc_full, 1);
        mbar_init(&p_ready, 128);
        mbar_init(&o_inter, 1);
        mbar_init(&o_scaled, 128);
        mbar_init(&o_full, 1);
        mbar_init(&o_free, 128);
        mbar_init(&s_full, 1);
        mbar_init(&s_conv, 128);
        mbar_init(&yt_ready, kYtThreads);
        mbar_init(&yt_done, 1);
        mbar_init(&fin[0], 1);
        mbar_init(&fin[1], 1);
        fence_barrier_init();
    }
    for (int i = threadIdx.x; i <= C; i += kMainThreads) pw[i] = exp2f(l2 * i);
    // powers that the tokens of a chunk have ahead of them: full chunks, and the short one
    for (int i = threadIdx.x; i < 2 * C; i += kMainThreads) {
        const int j = i % C, v = i < C ? C : vlast;
        wtab[i / C][j] = j < v ? exp2f(l2 * (rev ? j : v - 1 - j)) : 0.f;
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_base;
    const int items = nchunk * reps;

    if (warp == 0) {
        // ---------------- TMA producer: x tiles and y, z tiles in the order of their first use
        int nx = 0, ny = 0;
        bool ok = true;
        for (int k = 0; ok && k < nchunk; ++k) {
            const int c0 = chunk0(k);
            for (int r = 0; ok && r < reps; ++r) {
                const int hq = h * reps + r;
                if (r == 0 || many) {
                    const int s = ny % NY;
                    if (ny >= NY && !warp_wait(&yz_empty[s], (ny / NY - 1) & 1, &abort_flag)) { ok = false; break; }
                    uint8_t *y = yzbuf + s * K::YZ_BYTES, *z = y + K::Y_BYTES;
                    const int hyz = many ? hq : h;
                    mbar_arrive_expect_tx_w(&yz_full[s], K::YZ_BYTES);
                    for (int blk = 0; blk < DX / 64; ++blk) tma_load_4d_w(y + blk * C * 128, my, &yz_full[s], blk * 64, c0, hyz, b);
                    for (int blk = 0; blk < DZ / 64; ++blk) tma_load_4d_w(z + blk * C * 128, mz, &yz_full[s], blk * 64, c0, hyz, b);
                    ++ny;
                }
                if (r == 0 || !many) {
                    const int s = nx % NX;
                    if (nx >= NX && !warp_wait(&x_empty[s], (nx / NX - 1) & 1, &abort_flag)) { ok = false; break; }
                    uint8_t *x = xbuf + s * K::X_BYTES;
                    mbar_arrive_expect_tx_w(&x_full[s], C * DX * 2);
                    for (int blk = 0; blk < DX / 64; ++blk)
                        tma_load_4d_w(x + blk * C * 128, mx, &x_full[s], blk * 64, c0, many ? h : hq, b);
                    ++nx;
                }
            }
        }
        for (int i = nx > NX ? nx - NX : 0; i < nx; ++i) warp_drain(&x_full[i % NX], (i / NX) & 1);
        for (int i = ny > NY ? ny - NY : 0; i < ny; ++i) warp_drain(&yz_full[i % NY], (i / NY) & 1);
    } else if (warp == 1) {
        // ---------------- scores and P Z
        constexpr uint32_t idA = idesc_bf16(128, C, false, false);
        constexpr uint32_t idO = idesc_bf16(128, DZ, false, true);
        const uint32_t tO = tm + K::T_O, tA = tm + K::T_A;
        int ix = 0, iy = 0, ot = 0, k = 0, r = 0;   // x tile, y z tile, output tile, chunk, head
        for (int it = 0; it < items; ++it) {
            const bool first = r == 0, last = r == reps - 1;
            if ((first || !many) && !warp_wait(&x_full[ix % NX], (ix / NX) & 1, &abort_flag)) break;
            if ((first || many) && !warp_wait(&yz_full[iy % NY], (iy / NY) & 1, &abort_flag)) break;
            const uint32_t x = smem_u32(xbuf + (ix % NX) * K::X_BYTES);
            const uint32_t y = smem_u32(yzbuf + (iy % NY) * K::YZ_BYTES), z = y + K::Y_BYTES;
            tc_fence_after();
            LA_TL(it, 0);
            // (P of the item before has been read: this warp's MMAs run in the order of their issue)
#pragma unroll
            for (int kk = 0; kk < DX / 16; ++kk) mma_bf16_w(tA, desc_kmajor(x, C, 0, kk), desc_kmajor(y, C, 0, kk), idA, kk > 0);
            mma_commit_w(&sc_full);
            LA_TL(it, 1);
            if ((first || !many) && !warp_wait(&o_scaled, ot & 1, &abort_flag)) break;
            LA_TL(it, 5);
            // rows past a sequence's length are zeroed by the Y^T warps before P Z may read them (o_scaled says
            // that every earlier Y^T is over)
            if (p.lengths && first && k == nchunk - 1 && vlast < C && !warp_wait(&yt_ready, k & 1, &abort_flag)) break;
            if (!warp_wait(&p_ready, it & 1, &abort_flag)) break;
            LA_TL(it, 4);
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < C / 16; ++kk) mma_bf16_ta_w(tO, tA + kk * 8, desc_mnmajor(z, C, 0, kk), idO, 1u);
            if (last || !many) {
                mma_commit_w(&o_full);
                ++ot;
                ++ix;
            }
            if (last || many) {
                mma_commit_w(&yz_empty[iy % NY]);
                ++iy;
            }
            LA_TL(it, 6);
            if (++r == reps) {
                r = 0;
                ++k;
            }
        }
        mma_commit_w(&fin[0]);
        warp_drain(&fin[0], 0);
    } else if (warp == 2) {
        // ---------------- X S_bf, once for each output tile, and S += Y^T Z, once for each y z tile (grouped queries:
        // after the chunk's last X S_bf)
        constexpr uint32_t idO = idesc_bf16(128, DZ, false, true);
        const uint32_t sb = smem_u32(sbf), tS = tm + K::T_S, tO = tm + K::T_O;
        const uint32_t tYh = tm + K::T_YH, tYl = tm + K::T_YL;
        int ix = 0, iy = 0, k = 0, r = 0;
        for (int it = 0; it < items; ++it) {
            const bool first = r == 0, last = r == reps - 1;
            if (first || !many) {
                if (!warp_wait(&x_full[ix % NX], (ix / NX) & 1, &abort_flag)) break;
                if (first && !warp_wait(&s_conv, k & 1, &abort_flag)) break;
                if (ix > 0 && !warp_wait(&o_free, (ix - 1) & 1, &abort_flag)) break;
                LA_TL(it, 2);
                tc_fence_after();
                const uint32_t x = smem_u32(xbuf + (ix % NX) * K::X_BYTES);
#pragma unroll
                for (int kk = 0; kk < DX / 16; ++kk)
                    mma_bf16_w(tO, desc_kmajor(x, C, 0, kk), desc_mnmajor(sb, DX, 0, kk), idO, kk > 0);
                mma_commit_w(&o_inter);
                ++ix;
            }
            if (last || many) {
                if (!warp_wait(&yt_ready, iy & 1, &abort_flag)) break;
                LA_TL(it, 3);
                tc_fence_after();
                const uint32_t z = smem_u32(yzbuf + (iy % NY) * K::YZ_BYTES) + K::Y_BYTES;
#pragma unroll
                for (int kk = 0; kk < C / 16; ++kk) {
                    mma_bf16_ta_w(tS, tYh + kk * 8, desc_mnmajor(z, C, 0, kk), idO, 1u);
                    mma_bf16_ta_w(tS, tYl + kk * 8, desc_mnmajor(z, C, 0, kk), idO, 1u);
                }
                mma_commit_w(&yt_done);
                if (last) mma_commit_w(&s_full);
                mma_commit_w(&yz_empty[iy % NY]);
                ++iy;
            }
            if (++r == reps) {
                r = 0;
                ++k;
            }
        }
        mma_commit_w(&fin[1]);
        warp_drain(&fin[1], 0);
    } else if (warp >= 4 && warp < 8) {
        // ---------------- P = bf16(A o W), thread = row i, 16 columns at a time.  Away from the diagonal
        // gamma^|i - j| = gamma^(distance to the block's near end) gamma^(distance in the block), the latter in registers
        const int wq = warp % 4, i = wq * 32 + threadIdx.x % 32;
        const uint32_t ta = tm + K::T_A + ((uint32_t)(wq * 32) << 16);
        float g[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) g[e] = pw[rev ? e : 15 - e];
        for (int it = 0; it < items; ++it) {
            if (!warp_wait(&sc_full, it & 1, &abort_flag)) break;
            tc_fence_after();
            if (i == 127) LA_TL(it, 7);
#pragma unroll 1
            for (int cb = 0; cb < C / 32; ++cb) {
                uint32_t w[16];
                if (rev ? cb < wq : cb > wq) {   // the warp's rows have no such token
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = 0u;
                } else {
                    float v[32];
                    tmem_ld32(ta + cb * 32, v);
                    tmem_wait_regs<32>(v);
#pragma unroll
                    for (int hb = 0; hb < 2; ++hb) {
                        const int j0 = cb * 32 + hb * 16;
                        if (cb == wq) {   // the diagonal: tokens on this side of it
                            const float ago0 = (float)(rev ? j0 - i : i - j0);
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float ago = ago0 + (rev ? (float)e : -(float)e);
                                float x;
                                asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(ago * l2));
                                v[hb * 16 + e] = ago >= 0.f ? v[hb * 16 + e] * x : 0.f;
                            }
                        } else {
                            const float base = pw[rev ? j0 - i : i - j0 - 15];
#pragma unroll
                            for (int e = 0; e < 16; e += 2) {
                                float a = g[e], b = g[e + 1];
                                mul2(a, b, base, base);
                                mul2(v[hb * 16 + e], v[hb * 16 + e + 1], a, b);
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
                }
                // over the scores of this row that have been read (columns 16 cb .. 16 cb + 15 <= 32 cb + 31)
                tmem_st16_raw(ta + cb * 16, w);
            }
            tmem_st_wait();
            tc_fence_before();
            if (i == 127) LA_TL(it, 8);
            mbar_arrive_warp(&p_ready);
        }
    } else if (warp >= 8 && warp < 12) {
        // ---------------- S: the operand S_bf of the state before the chunk, and its decay; thread = row d
        const int wq = warp % 4, d = wq * 32 + threadIdx.x % 32;
        const uint32_t ts = tm + K::T_S + ((uint32_t)(wq * 32) << 16);
        const bool have = wq * 32 < DX;
        const size_t E = (size_t)p.D * p.Dv;
        // the segment's starting state (element [d][e] of the pass's state is at d sd + e se of a stored one)
        const size_t sd = ps.tr ? 1 : p.Dv, se = ps.tr ? p.Dv : 1;
        const float *from = p.nseg > 1 ? ps.slots + (size_t)bg * p.nseg * E : ps.init ? ps.init + (size_t)bg * E : nullptr;
        const float m0 = p.nseg > 1 ? (u > 0 ? exp2f(l2 * (part.before - ps.first_off)) : 1.f) : ps.init_mul;
        auto start16 = [&](int e0, float *v) {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = 0.f;
            if (!from) return;
            const float *f = from + d * sd + e0 * se;
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = f[e * se] * m0;
            for (int w = 1; w <= u; ++w) {
                const float g = exp2f(l2 * (part.before - (part_of(n, p.N, w, p.nseg, p.seg_len, rev).before)));
                if (g == 0.f) continue;   // decayed to nothing
                const float *fw = f + (size_t)w * E;
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = fmaf(fw[e * se], g, v[e]);
            }
        };
        bool ok = true;
        for (int k = 0; k < nchunk; ++k) {
            const int valid = min(C, part.hi - chunk0(k));
            const float g = pw[valid - (k == 0 ? off0 : 0)];
            if (k > 0) {
                ok = warp_wait(&s_full, (k - 1) & 1, &abort_flag);
                if (!ok) break;
                tc_fence_after();
            }
            if (d == 0) LA_TL(k, 9);
            if (have) {
#pragma unroll 1
                for (int c32 = 0; c32 < DZ / 32; ++c32) {
                    float v[32];
                    if (k == 0) {
                        start16(c32 * 32, v);
                        start16(c32 * 32 + 16, v + 16);
                    } else {
                        tmem_ld32(ts + c32 * 32, v);
                        tmem_wait_regs<32>(v);
                    }
                    store_state_row<DX>(sbf, d, v, 2 * c32);
                    store_state_row<DX>(sbf, d, v + 16, 2 * c32 + 1);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) mul2(v[e], v[e + 1], g, g);
                    tmem_st16(ts + c32 * 32, v);
                    tmem_st16(ts + c32 * 32 + 16, v + 16);
                }
                tmem_st_wait();
            }
            fence_proxy_async();
            tc_fence_before();
            if (d == 0) LA_TL(k, 10);
            mbar_arrive_warp(&s_conv);
        }
        if (ok && ps.fin && u == p.nseg - 1) {
            // what leaves a reverse pass decays once more; with no token at all it is what came in
            const float mul = ps.fin_mul * (ps.first_off && n > 0 ? exp2f(l2 * ps.first_off) : 1.f);
            if (nchunk > 0) {
                ok = warp_wait(&s_full, (nchunk - 1) & 1, &abort_flag);
                tc_fence_after();
            }
            float *f = ps.fin + (size_t)bg * E + d * sd;
            if (ok && have)
#pragma unroll 1
                for (int c16 = 0; c16 < DZ / 16; ++c16) {
                    float v[16];
                    if (nchunk > 0) {
                        tmem_ld16(ts + c16 * 16, v);
                        tmem_wait_regs<16>(v);
                    } else {
                        start16(c16 * 16, v);
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) f[(size_t)(c16 * 16 + e) * se] = v[e] * mul;
                }
        }
    } else if (warp >= 12 && warp < 16) {
        // ---------------- O: row i of X S_bf times gamma^(i + 1), then the finished tile to memory; thread = row i
        const int wq = warp % 4, i = wq * 32 + threadIdx.x % 32;
        const uint32_t to = tm + K::T_O + ((uint32_t)(wq * 32) << 16);
        const int tiles = many ? nchunk : items;
        int k = 0, r = 0;
        for (int t = 0; t < tiles; ++t) {
            const int c0 = chunk0(k), valid = min(C, part.hi - c0);
            const int hx = many ? h : h * reps + r;
            if (!warp_wait(&o_inter, t & 1, &abort_flag)) break;
            tc_fence_after();
            if (i == 0) LA_TL(t, 11);
            const float g = pw[max((rev ? valid - i : i + 1) - (k == 0 ? off0 : 0), 0)];
#pragma unroll 1
            for (int c32 = 0; c32 < DZ / 32; ++c32) {
                float v[32];
                tmem_ld32(to + c32 * 32, v);
                tmem_wait_regs<32>(v);
#pragma unroll
                for (int e = 0; e < 32; e += 2) mul2(v[e], v[e + 1], g, g);
                tmem_st16(to + c32 * 32, v);
                tmem_st16(to + c32 * 32 + 16, v + 16);
            }
            tmem_st_wait();
            tc_fence_before();
            if (i == 0) LA_TL(t, 12);
            mbar_arrive_warp(&o_scaled);
            if (!warp_wait(&o_full, t & 1, &abort_flag)) break;
            tc_fence_after();
            if (i == 0) LA_TL(t, 13);
            // staged in the x tile, which no MMA reads any more; rows past the length are zeros
            uint8_t *o = xbuf + (t % NX) * K::X_BYTES;
            const uint32_t keep = i < valid ? ~0u : 0u;
#pragma unroll 1
            for (int c32 = 0; c32 < DZ / 32; ++c32) {
                float v[32];
                tmem_ld32(to + c32 * 32, v);
                tmem_wait_regs<32>(v);
#pragma unroll
                for (int e = 0; e < 32; e += 2) mul2(v[e], v[e + 1], p.scale, p.scale);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = pack_bf16x2(v[8 * q + 2 * e], v[8 * q + 2 * e + 1]) & keep;
                    *reinterpret_cast<uint4 *>(o + swz_chunk(C, i, c32 * 4 + q)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            tc_fence_before();
            mbar_arrive_warp(&o_free);
            fence_proxy_async();
            __syncwarp();
            if (c0 + wq * 32 < p.N)
                for (int blk = 0; blk < DZ / 64; ++blk)
                    tma_store_4d_w(mo, o + blk * C * 128 + wq * 32 * 128, blk * 64, c0 + wq * 32, hx, b);
            bulk_commit();
            bulk_wait_read();
            mbar_arrive_w(&x_empty[t % NX]);
            if (i == 0) LA_TL(t, 14);
            if (many || ++r == reps) {
                r = 0;
                ++k;
            }
        }
        bulk_wait_all();
    } else if (warp >= 16) {
        // ---------------- Y^T of every y z tile; thread = (half of the tokens, lane d)
        const int wq = warp % 4, half = (warp - 16) / 4;
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        const int tiles = many ? items : nchunk;
        YtWeights w;
        bool shorter = false;
        for (int t = 0; t < tiles; ++t) {
            const int k = many ? t / reps : t, c0 = chunk0(k), valid = min(C, part.hi - c0);
            if (!warp_wait(&yz_full[t % NY], (t / NY) & 1, &abort_flag)) break;
            uint8_t *y = yzbuf + (t % NY) * K::YZ_BYTES;
            if (p.lengths && valid < C) {
                zero_rows<DZ>(y + K::Y_BYTES, valid, threadIdx.x - 512, kYtThreads);
                fence_proxy_async();
            }
            if (t > 0 && !warp_wait(&yt_done, (t - 1) & 1, &abort_flag)) break;
            tc_fence_after();
            if (wq * 32 < DX) {
                if (t == 0 || (valid < C) != shorter) {
                    shorter = valid < C;
                    w.set(&wtab[shorter][half * 64], 1.f);
                }
                yt_block(y, wq * 32, half * 64, w, valid, tm + K::T_YH + lane_off + half * 32, tm + K::T_YL + lane_off + half * 32);
                tmem_st_wait();
            }
            tc_fence_before();
            if (threadIdx.x == 512) LA_TL(t, 15);
            mbar_arrive_warp(&yt_ready);
        }
    }
    // rows of whole chunks past the sequence's length: zeros
    if (p.lengths) {
        const int z0 = max(part.lo + nchunk * C, u * p.seg_len), z1 = min(p.N, (u + 1) * p.seg_len);
        const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
        const int Hx = many ? p.Hkv : p.Hkv * reps;
        for (int r = 0; r < (many ? 1 : reps); ++r) {
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(ps.out) + ((size_t)b * Hx + (many ? h : h * reps + r)) * p.N * DZ;
            for (long long idx = threadIdx.x; idx < (long long)(z1 - z0) * (DZ / 8); idx += kMainThreads)
                *reinterpret_cast<uint4 *>(o + (size_t)(z0 + idx / (DZ / 8)) * DZ + idx % (DZ / 8) * 8) = zero;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tm, 512);
    if (threadIdx.x == 0 && abort_flag) atomicExch(p.err, kErrTimeout);
}

// ---------------------------------------------------------------------------------------
// The sums over single segments (see DecayStateParams).  Y^T is decayed to the segment's end at once, so S in
// TMEM only ever accumulates; Y^T is double-buffered and made by two groups of warps in turn.
// Warps: 0 TMA, 1 MMA, 4-11 and 12-19 Y^T of even and odd tiles (4-7 then write S).
constexpr int kStateThreads = 640;

struct StateMaps {
    CUtensorMap m[2][2];   // per array: y, z
};

template <int D, int DV>
struct StateCfg {
    static constexpr int Y_BYTES = C * D * 2, STAGE = Y_BYTES + C * DV * 2;
    static constexpr int NS = (kSmemLimit - 1024 - 2048) / STAGE > 4 ? 4 : (kSmemLimit - 1024 - 2048) / STAGE;
    static constexpr int SMEM = NS * STAGE + 1024;
};

template <int D, int DV>
__global__ void __launch_bounds__(kStateThreads, 1) k_decay_tc_state(const __grid_constant__ StateMaps maps,
                                                                     const __grid_constant__ DecayStateParams p) {
    using K = StateCfg<D, DV>;
    constexpr int NS = K::NS;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[NS], empty[NS], yt_ready[2], yt_done[2], fin;
    __shared__ __align__(16) float wtab[2][C];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    uint8_t *stage = align1024(smem_raw);
    pdl_wait();
    const int warp = threadIdx.x / 32;
    const int u = blockIdx.x % (p.nseg - 1), ah = blockIdx.x / (p.nseg - 1);
    const int a = ah / (p.B * p.Hkv), bg = ah % (p.B * p.Hkv), b = bg / p.Hkv, h = bg % p.Hkv;
    const int n = decay_tokens(p.lengths, b, p.N), rev = p.rev[a], heads = p.heads[a];
    const Part part = part_of(n, p.N, u, p.nseg, p.seg_len, rev);
    const int nchunk = (part.hi - part.lo + C - 1) / C, items = nchunk * heads;
    const float l2 = decay_log2(p.log_decay[h]);
    const int vlast = part.hi - part.lo - C * (nchunk - 1);
    const size_t E = (size_t)D * DV;
    float *slots = p.slots[a] + (size_t)bg * p.nseg * E;

    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&yt_ready[s], kYtThreads);
            mbar_init(&yt_done[s], 1);
        }
        mbar_init(&fin, 1);
        fence_barrier_init();
    }
    for (int i = threadIdx.x; i < 2 * C; i += kStateThreads) {
        const int j = i % C, v = i < C ? C : vlast;
        wtab[i / C][j] = j < v ? exp2f(l2 * (rev ? j : v - 1 - j)) : 0.f;
    }
    if (warp == 1) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_base;
    constexpr int T_S = 0, T_Y = 128;   // buffer i: hi at T_Y + 128 i, lo 64 further

    if (warp == 0) {
        int issued = 0;
        for (int it = 0; it < items; ++it) {
            const int s = it % NS, c0 = part.lo + C * (it / heads), hh = h * heads + it % heads;
            if (it >= NS && !warp_wait(&empty[s], (it / NS - 1) & 1, &abort_flag)) break;
            uint8_t *y = stage + s * K::STAGE, *z = y + K::Y_BYTES;
            mbar_arrive_expect_tx_w(&full[s], K::STAGE);
            for (int blk = 0; blk < D / 64; ++blk) tma_load_4d_w(y + blk * C * 128, &maps.m[a][0], &full[s], blk * 64, c0, hh, b);
            for (int blk = 0; blk < DV / 64; ++blk) tma_load_4d_w(z + blk * C * 128, &maps.m[a][1], &full[s], blk * 64, c0, hh, b);
            issued = it + 1;
        }
        for (int i = issued > NS ? issued - NS : 0; i < issued; ++i) warp_drain(&full[i % NS], (i / NS) & 1);
    } else if (warp == 1) {
        constexpr uint32_t id = idesc_bf16(128, DV, false, true);
        for (int it = 0; it < items; ++it) {
            const int s = it % NS, q = it % 2;
            if (!warp_wait(&yt_ready[q], (it / 2) & 1, &abort_flag)) break;
            tc_fence_after();
            const uint32_t z = smem_u32(stage + s * K::STAGE + K::Y_BYTES), ty = tm + T_Y + 128 * q;
            for (int kk = 0; kk < C / 16; ++kk) {
                mma_bf16_ta_w(tm + T_S, ty + kk * 8, desc_mnmajor(z, C, 0, kk), id, it > 0 || kk > 0);
                mma_bf16_ta_w(tm + T_S, ty + 64 + kk * 8, desc_mnmajor(z, C, 0, kk), id, 1u);
            }
            mma_commit_w(&yt_done[q]);
            mma_commit_w(&empty[s]);
        }
        mma_commit_w(&fin);
        warp_drain(&fin, 0);
    } else if (warp >= 4) {
        const int grp = (warp - 4) / 8, wq = warp % 4, half = ((warp - 4) / 4) % 2, d = wq * 32 + threadIdx.x % 32;
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        bool ok = true;
        for (int it = grp; it < items; it += 2) {
            const int s = it % NS, c0 = part.lo + C * (it / heads), valid = min(C, part.hi - c0), q = it % 2;
            // the buffer's last tile first: then every earlier use of this stage is over too (a group sees
            // only every other tile, and a parity tells only neighbouring phases apart)
            if (it >= 2 && !(ok = warp_wait(&yt_done[q], (it / 2 - 1) & 1, &abort_flag))) break;
            if (!(ok = warp_wait(&full[s], (it / NS) & 1, &abort_flag))) break;
            uint8_t *y = stage + s * K::STAGE;
            if (p.lengths && valid < C) {
                zero_rows<DV>(y + K::Y_BYTES, valid, (threadIdx.x - 128) % kYtThreads, kYtThreads);
                fence_proxy_async();
            }
            tc_fence_after();
            if (wq * 32 < D) {
                // what the chunk's last token has ahead of it in the segment
                YtWeights w;
                w.set(&wtab[valid < C][half * 64], exp2f(l2 * (rev ? c0 - part.lo : part.hi - c0 - valid)));
                yt_block(y, wq * 32, half * 64, w, valid, tm + T_Y + 128 * q + lane_off + half * 32,
                         tm + T_Y + 128 * q + 64 + lane_off + half * 32);
                tmem_st_wait();
            }
            tc_fence_before();
            mbar_arrive_warp(&yt_ready[q]);
        }
        if (warp < 8 && wq * 32 < D) {
            if (ok && items > 0) ok = warp_wait(&fin, 0, &abort_flag);
            tc_fence_after();
            if (ok)
#pragma unroll 1
                for (int c16 = 0; c16 < DV / 16; ++c16) {
                    float v[16];
                    if (items > 0) {
                        tmem_ld16(tm + T_S + lane_off + c16 * 16, v);
                        tmem_wait_regs<16>(v);
                    } else {
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[e] = 0.f;
                    }
                    float4 *f = reinterpret_cast<float4 *>(slots + (size_t)(u + 1) * E + (size_t)d * DV + c16 * 16);
#pragma unroll
                    for (int e = 0; e < 4; ++e) f[e] = make_float4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
                }
        } else if (warp >= 12 && u == 0) {   // slot 0: the starting state
            const float *f = p.init[a] ? p.init[a] + (size_t)bg * E : nullptr;
            for (int i = threadIdx.x - 384; i < (int)E; i += 256) slots[i] = f ? f[i] * p.init_mul[a] : 0.f;
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tm, 512);
    if (threadIdx.x == 0 && abort_flag) atomicExch(p.err, kErrTimeout);
}

// ---- launches ---------------------------------------------------------------------------

Strides out_strides(int H, int N, int W) { return contiguous_strides(H, N, W); }

template <int DX, int DZ>
cudaError_t passes_d(const DecayParams &p, int pass0, int npass, cudaStream_t s) {
    PassMaps maps;
    for (int i = pass0; i < pass0 + npass; ++i) {
        const DecayPass &ps = p.pass[i];
        const int Hq = p.Hkv * p.n_rep, Hx = ps.many_yz ? p.Hkv : Hq, Hyz = ps.many_yz ? Hq : p.Hkv;
        cudaError_t e = make_map_in(&maps.m[i][0], ps.x, p.B, Hx, p.N, DX, ps.sx, C);
        if (e == cudaSuccess) e = make_map_in(&maps.m[i][1], ps.y, p.B, Hyz, p.N, DX, ps.sy, C);
        if (e == cudaSuccess) e = make_map_in(&maps.m[i][2], ps.z, p.B, Hyz, p.N, DZ, ps.sz, C);
        if (e == cudaSuccess) e = make_map_in(&maps.m[i][3], ps.out, p.B, Hx, p.N, DZ, out_strides(Hx, p.N, DZ), 32);
        if (e != cudaSuccess) return e;
    }
    auto kern = k_decay_tc<DX, DZ>;
    cudaError_t e = prepare(kern, MainCfg<DX, DZ>::SMEM);
    if (e != cudaSuccess) return e;
    TraceScope tr("decay_tc", s);
    return launch_pdl(kern, dim3((unsigned)npass * p.nseg * p.B * p.Hkv), dim3(kMainThreads), MainCfg<DX, DZ>::SMEM, s, maps,
                      p, pass0, npass);
}

cudaError_t passes(const DecayParams &p, int pass0, int npass, cudaStream_t s) {
    const bool tr = p.pass[pass0].tr;
    const int DX = tr ? p.Dv : p.D, DZ = tr ? p.D : p.Dv;
    if (DX == 64) return DZ == 64 ? passes_d<64, 64>(p, pass0, npass, s) : passes_d<64, 128>(p, pass0, npass, s);
    return DZ == 64 ? passes_d<128, 64>(p, pass0, npass, s) : passes_d<128, 128>(p, pass0, npass, s);
}

template <int D, int DV>
cudaError_t states_d(const DecayStateParams &p, cudaStream_t s) {
    StateMaps maps;
    for (int a = 0; a < p.n; ++a) {
        cudaError_t e = make_map_in(&maps.m[a][0], p.y[a], p.B, p.Hkv * p.heads[a], p.N, D, p.sy[a], C);
        if (e == cudaSuccess) e = make_map_in(&maps.m[a][1], p.z[a], p.B, p.Hkv * p.heads[a], p.N, DV, p.sz[a], C);
        if (e != cudaSuccess) return e;
    }
    auto kern = k_decay_tc_state<D, DV>;
    cudaError_t e = prepare(kern, StateCfg<D, DV>::SMEM);
    if (e != cudaSuccess) return e;
    TraceScope tr("decay_tc_state", s);
    return launch_pdl(kern, dim3((unsigned)p.n * (p.nseg - 1) * p.B * p.Hkv), dim3(kStateThreads), StateCfg<D, DV>::SMEM, s,
                      maps, p);
}

}  // namespace

cudaError_t decay_tc_states(const DecayStateParams &p, cudaStream_t s) {
    if (p.D == 64) return p.Dv == 64 ? states_d<64, 64>(p, s) : states_d<64, 128>(p, s);
    return p.Dv == 64 ? states_d<128, 64>(p, s) : states_d<128, 128>(p, s);
}

cudaError_t decay_tc_passes(const DecayParams &p, cudaStream_t s) {
    // the gradients' passes have two shapes of state, D x Dv and its transpose
    if (p.npass == 1 || p.D == p.Dv) return passes(p, 0, p.npass, s);
    cudaError_t e = passes(p, 0, 2, s);
    return e == cudaSuccess ? passes(p, 2, 1, s) : e;
}

}  // namespace la

#ifdef LA_TIMELINE
extern "C" int la_timeline_read_decay(long long *out) {
    return cudaMemcpyFromSymbol(out, la::g_la_tl, sizeof(long long) * 64 * 16) == cudaSuccess ? 0 : 1;
}
#endif
