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
// Warps: 0 TMA, 1 MMA, 4-7 P, 8-11 S -> S_bf and the decay of S, 12-15 O's row powers and the output,
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

// Y^T of one tile for the threads of lane quarter `wq`: lane d's 32 values j0 .. j0 + 31 times w[j] (times
// `mul`), as two bf16 terms into 16 columns each at th and tl.  Values at j >= valid are taken as zeros.
__device__ __forceinline__ void yt_block(const uint8_t *y, int d, int j0, const float *w, float mul, int valid,
                                         uint32_t th, uint32_t tl) {
    uint32_t hi[16], lo[16];
#pragma unroll
    for (int e = 0; e < 16; ++e) {
        const int j = j0 + 2 * e;
        uint32_t a = *reinterpret_cast<const uint16_t *>(y + swz_offset(C, j, d));
        uint32_t b = *reinterpret_cast<const uint16_t *>(y + swz_offset(C, j + 1, d));
        if (valid < C) {
            a = j < valid ? a : 0u;
            b = j + 1 < valid ? b : 0u;
        }
        const float2 wj = *reinterpret_cast<const float2 *>(w + j);
        const float fa = __uint_as_float(a << 16) * (wj.x * mul), fb = __uint_as_float(b << 16) * (wj.y * mul);
        const uint32_t h = pack_bf16x2(fa, fb);
        hi[e] = h;
        lo[e] = pack_bf16x2(fa - __uint_as_float(h << 16), fb - __uint_as_float(h & 0xffff0000u));
    }
    tmem_st16_raw(th, hi);
    tmem_st16_raw(tl, lo);
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
    __shared__ uint64_t sc_full, p_ready, o_inter, o_scaled, o_full, o_free, s_full, s_conv, yt_ready, yt_done, fin;
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
            mbar_init(&yz_empty[s], 1);
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
        mbar_init(&fin, 1);
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
        // ---------------- MMA issuer
        constexpr uint32_t idA = idesc_bf16(128, C, false, false);
        constexpr uint32_t idO = idesc_bf16(128, DZ, false, true);
        const uint32_t sb = smem_u32(sbf), tS = tm + K::T_S, tO = tm + K::T_O, tA = tm + K::T_A;
        const uint32_t tYh = tm + K::T_YH, tYl = tm + K::T_YL;
        int ix = 0, iy = 0, st = 0, ot = 0;   // x tile, y z tile, state update, output tile
        bool ok = true;
        for (int it = 0; ok && it < items; ++it) {
            const int k = it / reps, r = it % reps;
            const bool first = r == 0, last = r == reps - 1;
            if (first || !many) {
                if (it > 0) ++ix;
                if (!warp_wait(&x_full[ix % NX], (ix / NX) & 1, &abort_flag)) break;
            }
            if (first || many) {
                if (it > 0) ++iy;
                if (!warp_wait(&yz_full[iy % NY], (iy / NY) & 1, &abort_flag)) break;
            }
            const uint32_t x = smem_u32(xbuf + (ix % NX) * K::X_BYTES);
            const uint32_t y = smem_u32(yzbuf + (iy % NY) * K::YZ_BYTES), z = y + K::Y_BYTES;
            tc_fence_after();
            // scores (P of the item before has been read: MMAs run in the order of their issue)
            for (int kk = 0; kk < DX / 16; ++kk) mma_bf16_w(tA, desc_kmajor(x, C, 0, kk), desc_kmajor(y, C, 0, kk), idA, kk > 0);
            mma_commit_w(&sc_full);
            // X S_bf, once for each output tile
            if (first || !many) {
                if (first && !warp_wait(&s_conv, k & 1, &abort_flag)) break;
                if (ot > 0 && !warp_wait(&o_free, (ot - 1) & 1, &abort_flag)) break;
                tc_fence_after();
                for (int kk = 0; kk < DX / 16; ++kk) mma_bf16_w(tO, desc_kmajor(x, C, 0, kk), desc_mnmajor(sb, DX, 0, kk), idO, kk > 0);
                mma_commit_w(&o_inter);
            }
            // S += Y^T Z, once for each y z tile (grouped queries: with the chunk's last head)
            const bool upd = many || last;
            // tiles with rows past the length are zeroed by the Y^T warps before P Z may read them (such
            // a tile is the sequence's last, of grouped queries: its Y^T serves the last head's update too)
            const bool zeroed = p.lengths && chunk0(k) + C > part.hi;
            if (zeroed ? first : upd) {
                if (!warp_wait(&yt_ready, st & 1, &abort_flag)) break;
                tc_fence_after();
            }
            if (upd) {
                for (int kk = 0; kk < C / 16; ++kk) {
                    mma_bf16_ta_w(tS, tYh + kk * 8, desc_mnmajor(z, C, 0, kk), idO, 1u);
                    mma_bf16_ta_w(tS, tYl + kk * 8, desc_mnmajor(z, C, 0, kk), idO, 1u);
                }
                mma_commit_w(&yt_done);
                if (last) mma_commit_w(&s_full);
                ++st;
            }
            // O += P Z
            if (!warp_wait(&p_ready, it & 1, &abort_flag)) break;
            if ((first || !many) && !warp_wait(&o_scaled, ot & 1, &abort_flag)) break;
            tc_fence_after();
            for (int kk = 0; kk < C / 16; ++kk) mma_bf16_ta_w(tO, tA + kk * 8, desc_mnmajor(z, C, 0, kk), idO, 1u);
            if (last || !many) {
                mma_commit_w(&o_full);
                ++ot;
            }
            if (upd) mma_commit_w(&yz_empty[iy % NY]);
        }
        mma_commit_w(&fin);
        warp_drain(&fin, 0);
    } else if (warp >= 4 && warp < 8) {
        // ---------------- P = bf16(A o W), thread = row i
        const int wq = warp % 4, lane = threadIdx.x % 32, i = wq * 32 + lane;
        const uint32_t ta = tm + K::T_A + ((uint32_t)(wq * 32) << 16);
        for (int it = 0; it < items; ++it) {
            if (!warp_wait(&sc_full, it & 1, &abort_flag)) break;
            tc_fence_after();
#pragma unroll 1
            for (int cb = 0; cb < C / 32; ++cb) {
                uint32_t w[16];
                if (rev ? cb < wq : cb > wq) {   // the warp's rows have no such token
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = 0u;
                } else {
                    float v[32];
                    tmem_ld32(ta + cb * 32, v);
                    if (cb == wq) {
                        // gamma^|i - j| of the tokens on this side of the diagonal
                        const float *pd = pw;
                        tmem_wait_regs<32>(v);
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const int ago = rev ? e - lane : lane - e;
                            v[e] = ago >= 0 ? v[e] * pd[max(ago, 0)] : 0.f;
                        }
                    } else {
                        // gamma^|i - j| = gamma^(distance to the block's near end) gamma^(distance in the block)
                        const float base = pw[rev ? cb * 32 - i : i - cb * 32 - 31];
                        const float4 *t4 = reinterpret_cast<const float4 *>(rev ? pw : &wtab[0][C - 32]);
                        tmem_wait_regs<32>(v);
#pragma unroll
                        for (int q = 0; q < 8; ++q) {
                            const float4 t = t4[q];
                            v[4 * q] *= base * t.x;
                            v[4 * q + 1] *= base * t.y;
                            v[4 * q + 2] *= base * t.z;
                            v[4 * q + 3] *= base * t.w;
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
            if (have) {
#pragma unroll 1
                for (int c16 = 0; c16 < DZ / 16; ++c16) {
                    float v[16];
                    if (k == 0) {
                        start16(c16 * 16, v);
                    } else {
                        tmem_ld16(ts + c16 * 16, v);
                        tmem_wait_regs<16>(v);
                    }
                    store_state_row<DX>(sbf, d, v, c16);
#pragma unroll
                    for (int e = 0; e < 16; ++e) v[e] *= g;
                    tmem_st16(ts + c16 * 16, v);
                }
                tmem_st_wait();
            }
            fence_proxy_async();
            tc_fence_before();
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
        for (int t = 0; t < tiles; ++t) {
            const int k = many ? t : t / reps, c0 = chunk0(k), valid = min(C, part.hi - c0);
            const int hx = many ? h : h * reps + t % reps;
            if (!warp_wait(&o_inter, t & 1, &abort_flag)) break;
            tc_fence_after();
            const float g = pw[max((rev ? valid - i : i + 1) - (k == 0 ? off0 : 0), 0)];
#pragma unroll 1
            for (int c32 = 0; c32 < DZ / 32; ++c32) {
                float v[32];
                tmem_ld32(to + c32 * 32, v);
                tmem_wait_regs<32>(v);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] *= g;
                tmem_st16(to + c32 * 32, v);
                tmem_st16(to + c32 * 32 + 16, v + 16);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive_warp(&o_scaled);
            if (!warp_wait(&o_full, t & 1, &abort_flag)) break;
            tc_fence_after();
            // staged in the x tile, which no MMA reads any more; rows past the length are zeros
            uint8_t *o = xbuf + (t % NX) * K::X_BYTES;
            const float sc = i < valid ? p.scale : 0.f;
#pragma unroll 1
            for (int c32 = 0; c32 < DZ / 32; ++c32) {
                float v[32];
                tmem_ld32(to + c32 * 32, v);
                tmem_wait_regs<32>(v);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = i < valid ? pack_bf16x2(v[8 * q + 2 * e] * sc, v[8 * q + 2 * e + 1] * sc) : 0u;
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
        }
        bulk_wait_all();
    } else if (warp >= 16) {
        // ---------------- Y^T of every y z tile; thread = (half of the tokens, lane d)
        const int wq = warp % 4, half = (warp - 16) / 4, d = wq * 32 + threadIdx.x % 32;
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        const int tiles = many ? items : nchunk;
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
#pragma unroll 1
                for (int q = 0; q < 2; ++q) {
                    const int j0 = half * 64 + q * 32;
                    yt_block(y, d, j0, wtab[valid < C], 1.f, valid, tm + K::T_YH + lane_off + j0 / 2, tm + K::T_YL + lane_off + j0 / 2);
                }
                tmem_st_wait();
            }
            tc_fence_before();
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
                const float mul = exp2f(l2 * (rev ? c0 - part.lo : part.hi - c0 - valid));
#pragma unroll 1
                for (int x = 0; x < 2; ++x) {
                    const int j0 = half * 64 + x * 32;
                    yt_block(y, d, j0, wtab[valid < C], mul, valid, tm + T_Y + 128 * q + lane_off + j0 / 2,
                             tm + T_Y + 128 * q + 64 + lane_off + j0 / 2);
                }
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
