// la_decay_tc.cu -- decayed linear attention on the tensor cores (tcgen05 / TMEM / TMA), bfloat16.
//
// One block walks one segment of one key/value head in chunks of C = 128 tokens.  Per chunk (X, Y, Z:
// see la_decay.cuh; W_ij = gamma^(i-j) for j <= i, else 0; scale gamma^(i+1) = 2^(e_i) m_i with 1 <= |m_i| < 2):
//   A  = X Y^T                                              [C x C]     scores
//   P  = bf16(scale A_ij W_ij / m_i)                        (fp32 decay, one rounding)
//   O  = P Z + (2^(e_i) x_i) (S_hi + S_lo)                  [C x DZ]    output row i: m_i O_i
//   S  = gamma^C S + bf16(gamma^(C-1-j) y_j)^T Z            [DX x DZ]   fp32 in TMEM
// Powers of gamma are only ever of whole distances >= 0, so no decay overflows.  Every term of an output is rounded
// to bf16 once on its way, besides the output itself: in P, or as the decayed y.  The x of a row takes a power of two
// only, which is exact (the rest of its decay waits for the float32 output, and P, rounded anyway, is made to fit), and S
// is read as two bf16 terms (2^-17).  So outputs are within sqrt(2) of what rounding them alone leaves (2.4e-3 against
// 1.7e-3 of the 2-norm); with x and S rounded once each they were at 3.1e-3 to 3.4e-3.  A state that goes out is not made
// here but by the state kernel below, in three terms.
//
// Operands made by the CUDA cores are read by the MMA from TMEM where it has room: P and the decayed X take the place
// of the scores (P over columns that its thread has read, the decayed X over the rest when P is done), Y^T has columns
// of its own.  That halves the MMA's shared-memory reads, which at 128 x 128 x 16 from shared memory would
// take all of its bandwidth, and leaves the shared memory to the TMA tiles.  The scores have two buffers, so that the
// next item's scores and P run beside this one's O; where S and O are 128 columns wide that takes Y^T's place, and y is
// decayed in its tile instead.
// Several heads of x share one chunk of y, z (grouped queries; S moves on after the last), or several heads
// of y, z share one of x (their gradients; O and S sum over the heads).
//
// Warps: 0 TMA of x, 3 of y and z, 1 MMA of scores and O, 2 MMA of S, 4-7 P, 8-11 S -> S_hi, S_lo and the decay of S,
// 12-15 the decayed X, 16-19 the output rows, 20-23 the decayed y (and the zeros past a sequence's length).
//
// The reverse passes (gradients of k and v) take the same steps with j >= i and gamma^(j-i), chunks from the
// last to the first.
//
// What bounds it: the chain of hand-overs from role to role, one block an SM: 2.5 us for a chunk and head of 128 x 128
// where y and z are shared (32 query on 8 heads, N 65536, D 128: 274 us, 108 of them a block), 3.1 us with one head each on
// every SM (8 x 19 heads, N 8192: 218 us; there the memory gives 6.4 TB/s), 2.0 us of 64 x 64.  The tensor pipe is busy
// for 16 to 39 % of the time, an SM's warps issue 1.1 to 1.8 instructions a cycle.  In copies of this kernel that leave out
// work (passes alone, us; gradients of 2 x 16 heads, N 8192, D 128 | 4 x 16, N 4096, D 64 | 32/8, N 65536, D 128): as it is
// 137 | 45 | 274; without the arithmetic of P 131 | 35 | 234, of the decayed X 133 | 43 | 252, of the decayed Y 137 | 45 |
// 256, of S 131 | 45 | 270; without the output's stores 131 | 45 | 270; without all of these 104 | 33 | 211; without most
// MMAs as well 90 | 31 | 160.  With x and S rounded to bf16 (and their MMA and tiles saved) it was 125 | 43 | 252.
#include "la_decay.cuh"
#include "la_tc_common.cuh"

namespace la {
namespace {

constexpr int C = kDecayTcChunk;
constexpr int kMainThreads = 768;

// Bounded warp-uniform wait.  A try suspends the thread for 2 us at most, so that kTries of them are a few seconds
// at most and tens of milliseconds at least; no wait of a block that runs takes one of them.  (The MMA warp of the scores
// polls two barriers in turn without a suspension, kTries times at most: tens of milliseconds.)  A role whose wait ran out
// leaves its loop, the others' waits then run out too, and the block ends as always: copies and MMAs in flight
// drained, TMEM freed, the error latched.
//
// Code size is what this and the loops below are shaped by.  Each role's loop body runs once a chunk, so the roles'
// code passes through the instruction caches in turn; at 38 KB in all it was fetched anew for each chunk (300
// misses of 128 bytes a chunk and SM, warps at one instruction in six cycles).  So a wait is a dozen instructions,
// loops stay rolled where that costs a few instructions, and there is one copy of each product.
#ifdef LA_TEST_HOOKS
constexpr uint32_t kTries = 1u << 13;
__device__ int g_la_test_skip_decay;   // withhold the first arrival of warp 4 of block 0: 1 passes, 2 sums (see there)
#else
constexpr uint32_t kTries = 1u << 21;
#endif
__device__ __forceinline__ bool await(uint64_t *bar, uint32_t parity, volatile int *abort) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 n;\n\tmov.b32 n, %3;\n"
        "AGAIN:\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 2000;\n\t"
        "@p bra OVER;\n\tsub.u32 n, n, 1;\n\tsetp.ne.u32 q, n, 0;\n\t@q bra AGAIN;\n"
        "OVER:\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity), "n"(kTries)
        : "memory");
    if (__all_sync(0xffffffffu, done)) return true;
    *abort = 1;
    return false;
}
__device__ __forceinline__ bool is_over(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_test(bar, parity));
}

// A place in a ring of stages and the parity of its current use.
struct Ring {
    int s = 0;
    uint32_t p = 0;
    __device__ __forceinline__ void next(int n) {
        if (++s == n) {
            s = 0;
            p ^= 1u;
        }
    }
};

struct PassMaps {
    CUtensorMap m[3][4];   // per pass: x, y, z, out
};

// YSM: y is decayed in place in shared memory (else Y^T is made in TMEM).
template <int DX, int DZ>
struct MainCfg {
    static constexpr bool YSM = DZ == 128;
    static constexpr int X_BYTES = C * DX * 2, Y_BYTES = C * DX * 2, Z_BYTES = C * DZ * 2, S_BYTES = DX * DZ * 2;
    static constexpr int O_BYTES = C * DZ * 2;
    // At 128 x 128 there is room for five tiles beside S: with several heads of x to one y, z (those are loaded once a
    // chunk) x has two stages, y one, z one and the output one; else x one (it is over when its scores are made and the row
    // factors' X is in registers), y and z two.
    static constexpr bool TIGHT = DX == 128 && DZ == 128;
    static constexpr int NX = DX == 64 ? (DZ == 64 ? 4 : 3) : 2;
    static constexpr int NY = DX == 64 ? 3 : 2;
    static constexpr int NZ = DX == 64 ? (DZ == 64 ? 4 : 3) : (DZ == 64 ? 3 : 2);
    // output tiles: of their own; with YSM in the z tile that is used up or, where several heads share it, in place of
    // y's other stages (which such a block needs less: a y tile serves all of them)
    static constexpr int NO = YSM ? 0 : DX == 64 ? 2 : 1;
    static constexpr int TILES = TIGHT ? 5 * X_BYTES : NX * X_BYTES + NY * Y_BYTES + NZ * Z_BYTES + NO * O_BYTES;
    static constexpr int SMEM = TILES + 2 * S_BYTES + 1024;
    static_assert(SMEM + 2048 <= kSmemLimit, "tiles, barriers and tables");
    static_assert(!YSM || (NY - 1) * Y_BYTES >= O_BYTES, "an output tile in y's other stages");
    // (S's MMA reads 128 columns from a y tile's start: with DX = 64 the next y stage or the first z tile)
    static_assert(DX == 128 || Z_BYTES >= C * 64 * 2, "128 columns from a y tile's start");
    // TMEM: S, O, two buffers of scores, Y^T
    static constexpr int NSC = 2;
    static constexpr int T_S = 0, T_O = DZ, T_A = 2 * DZ, T_Y = T_A + 128 * NSC;
    static_assert((YSM ? T_Y : T_Y + 64) <= 512, "TMEM columns");
};

// A block's part of the sequence: tokens [lo, hi).
struct Part {
    int lo, hi;
};
__device__ __forceinline__ Part part_of(int n, int N, int u, int nseg, int seg_len, int rev) {
    const int s = rev ? nseg - 1 - u : u;
    Part r;
    r.lo = min(n, s * seg_len);
    r.hi = min(n, r.lo + seg_len);
    return r;
}

// Part `sub` (in the pass's order) of segment u.
__device__ __forceinline__ Part sub_part_of(int n, int N, int u, int nseg, int seg_len, int sub, int nsub, int sub_len,
                                            int rev) {
    const int s = rev ? nseg - 1 - u : u, q = rev ? nsub - 1 - sub : sub;
    Part r;
    r.lo = min(n, s * seg_len + min(seg_len, q * sub_len));
    r.hi = min(n, s * seg_len + min(seg_len, (q + 1) * sub_len));
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

__device__ __forceinline__ void fma2(float &x, float &y, float a, float b, float c) {   // x = a c + x, y = b c + y
    unsigned long long p, q, r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(q) : "f"(a), "f"(b));
    asm("mov.b64 %0, {%1, %1};" : "=l"(r) : "f"(c));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(p) : "l"(q), "l"(r));
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
}

// The upper 8 bits of two floats' significands as bf16, taken off them: three of these are the whole 24.
__device__ __forceinline__ uint32_t cut_bf16x2(float2 &f) {
    const uint32_t x = __float_as_uint(f.x), y = __float_as_uint(f.y);
    fma2(f.x, f.y, __uint_as_float(x & 0xffff0000u), __uint_as_float(y & 0xffff0000u), -1.f);
    return __byte_perm(x, y, 0x7632);
}

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t u) { return *reinterpret_cast<__nv_bfloat162 *>(&u); }
__device__ __forceinline__ uint32_t as_u32(__nv_bfloat162 h) { return *reinterpret_cast<uint32_t *>(&h); }

// scale gamma^n of a row as 2^e and m (0 and 1 where it is nothing).
struct RowFactor {
    float p2, m;
};
__device__ __forceinline__ RowFactor row_factor(float f) {
    const uint32_t b = __float_as_uint(f), e = b & 0x7f800000u;
    RowFactor r;
    r.p2 = __uint_as_float(e);
    r.m = e ? __uint_as_float((b & 0x807fffffu) | 0x3f800000u) : 1.f;
    return r;
}

// The decays w of a chunk's tokens, 16 groups of 8 of which a thread meets 2 in each group, as two bf16
// terms.
struct YtWeights {
    uint32_t hi[16], lo[16];
    __device__ __forceinline__ void set(const float *w, float mul) {
#pragma unroll
        for (int g = 0; g < 16; ++g) {
            const float a = w[8 * g + 2 * (threadIdx.x % 4)] * mul, b = w[8 * g + 2 * (threadIdx.x % 4) + 1] * mul;
            hi[g] = pack_bf16x2(a, b);
            const float2 f = unpack_bf16x2(hi[g]);
            lo[g] = pack_bf16x2(a - f.x, b - f.y);
        }
    }
};

// Decayed Y^T of one tile for the warp's 32 lanes d from d0: y w in bf16 into 64 columns at th, with w = wh + wl (bf16
// each) as bf16(y wh + bf16(y wl)).  The tile's 8 x 8 blocks come transposed out of shared memory in the layout of the
// store.
__device__ __forceinline__ void yt_tile(const uint8_t *y, int d0, const YtWeights &w, uint32_t th) {
    const int t = threadIdx.x % 32;
#pragma unroll 1
    for (int half = 0; half < 2; ++half) {   // lanes d0 + 16 half ..
        const uint32_t addr = smem_u32(y) + swz_chunk(C, 8 * (t / 16) + t % 8, (d0 + 16 * half) / 8 + ((t / 8) & 1));
        const uint32_t lane = (uint32_t)(16 * half) << 16;
#pragma unroll
        for (int jq = 0; jq < 4; ++jq) {     // tokens 32 jq ..
            uint32_t v[8];
            ldmatrix_x4_trans(addr + jq * 32 * 128, v);
            ldmatrix_x4_trans(addr + (jq * 32 + 16) * 128, v + 4);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int g = jq * 4 + i / 2;   // group of 8 tokens
                const __nv_bfloat162 u = as_bf162(v[i]);
                v[i] = as_u32(__hfma2(u, as_bf162(w.hi[g]), __hmul2(u, as_bf162(w.lo[g]))));
            }
            tmem_st_frag16(th + lane + jq * 16, v);
        }
    }
}

// 16 columns of row d of S as two bf16 terms, into two tiles of D rows.
template <int D>
__device__ __forceinline__ void store_state_terms(uint8_t *hi, uint8_t *lo, int d, const float *v, int c16) {
    float r[16];
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
        const float2 h = unpack_bf16x2(pack_bf16x2(v[e], v[e + 1]));
        r[e] = v[e] - h.x;
        r[e + 1] = v[e + 1] - h.y;
    }
    store_state_row<D>(hi, d, v, c16);
    store_state_row<D>(lo, d, r, c16);
}

// Zero rows [valid, C) of a C x W tile (what lies past a sequence's length must not meet an MMA or a weight of
// 0, where 0 times a non-finite value is not 0); nth threads, this one being i.
template <int W>
__device__ __noinline__ void zero_rows(uint8_t *tile, int valid, int i, int nth) {
    for (int idx = i; idx < (C - valid) * (W / 8); idx += nth)
        *reinterpret_cast<uint4 *>(tile + swz_chunk(C, valid + idx / (W / 8), idx % (W / 8))) = make_uint4(0u, 0u, 0u, 0u);
}

template <int DX, int DZ>
__global__ void __launch_bounds__(kMainThreads, 1) k_decay_tc(const __grid_constant__ PassMaps maps,
                                                              const __grid_constant__ DecayParams p, int pass0,
                                                              int npass) {
    using K = MainCfg<DX, DZ>;
    constexpr bool YSM = K::YSM;
    constexpr int NXS = K::NX, NYS = K::NY, NZS = K::NZ, NSC = K::NSC, NO = K::NO;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t x_full[NXS], x_empty[NXS], y_full[NYS], y_empty[NYS], z_full[NZS], z_empty[NZS];
    // of one buffer of the scores: in, P made; by output tile: P of its first scores made, decayed X made
    __shared__ uint64_t sc_full[NSC], p_ready[NSC], p_first[2], xd_ready[2];
    __shared__ uint64_t y_scored[NYS], yt_ready[NYS];   // of a stage of y: its scores done, its decayed form made
    __shared__ uint64_t o_full, o_free, s_full, s_conv, yt_done, z_used[2], zeroed, fin[2];
    __shared__ __align__(16) float pw[C + 4], wtab[2][C];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    uint8_t *xbuf = align1024(smem_raw);
    pdl_wait();
    const int warp = threadIdx.x / 32;
    const int pi = pass0 + blockIdx.x % npass, rest = blockIdx.x / npass;
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < NXS; ++s) {
            mbar_init(&x_full[s], 1);
            mbar_init(&x_empty[s], 1 + 4);             // its scores' MMA, warps of the decayed X
        }
        for (int s = 0; s < NYS; ++s) {
            mbar_init(&y_full[s], 1);
            mbar_init(&y_empty[s], YSM ? 1 : 4 + 4);   // S's MMA, or warps of P, of Y^T
            mbar_init(&y_scored[s], 1);
            mbar_init(&yt_ready[s], 128);
        }
        for (int s = 0; s < NZS; ++s) {
            mbar_init(&z_full[s], 1);
            mbar_init(&z_empty[s], YSM ? 2 + 4 : 2);   // both MMA warps (and the warps that store the output)
        }
        for (int s = 0; s < NSC; ++s) {
            mbar_init(&sc_full[s], 1);
            mbar_init(&p_ready[s], 128);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(&p_first[s], 128);
            mbar_init(&xd_ready[s], 128);
        }
        mbar_init(&o_full, 1);
        mbar_init(&o_free, 128);
        mbar_init(&s_full, 2);
        mbar_init(&s_conv, 128);
        mbar_init(&yt_done, 1);
        mbar_init(&z_used[0], 1);
        mbar_init(&z_used[1], 1);
        mbar_init(&zeroed, 128);
        mbar_init(&fin[0], 1);
        mbar_init(&fin[1], 1);
        fence_barrier_init();
    }
    if (threadIdx.x >= 96 && threadIdx.x < 100) tma_prefetch_map(&maps.m[pi][threadIdx.x - 96]);
    if (warp == 1) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    const DecayPass &ps = p.pass[pi];
    const int heads = p.B * p.Hkv, bg = rest % heads, b = bg / p.Hkv, h = bg % p.Hkv;
    const int n = decay_tokens(p.lengths, b, p.N), rev = ps.rev, many = ps.many_yz, reps = p.n_rep;
    // (the last segment in token order may be a short one: those blocks come last)
    const int u = rev ? p.nseg - 1 - rest / heads : rest / heads;
    // stages in use; with YSM output tiles are staged in z's, or (shared y and z) in place of y's second
    const bool shared = !many && reps > 1, o_in_z = YSM && !shared;
    const int NX = K::TIGHT && !shared ? 1 : NXS, NY = YSM && shared ? 1 : NYS, NZ = K::TIGHT && shared ? 1 : NZS;
    uint8_t *ybuf = xbuf + NX * K::X_BYTES;
    uint8_t *zbuf = ybuf + NYS * K::Y_BYTES;
    uint8_t *sbf = xbuf + K::TILES, *slo = sbf + K::S_BYTES;
    uint8_t *obuf = YSM ? ybuf + K::Y_BYTES : zbuf + NZS * K::Z_BYTES;
    const Part part = part_of(n, p.N, u, p.nseg, p.seg_len, rev);
    const int nchunk = (part.hi - part.lo + C - 1) / C;
    const int off0 = u == 0 ? ps.first_off : 0;   // of the first chunk
    const float l2 = decay_log2(p.log_decay[h]);
    auto chunk0 = [&](int k) { return part.lo + C * (rev ? nchunk - 1 - k : k); };
    // tokens of the short chunk (the last in token order)
    const int vlast = part.hi - part.lo - C * (nchunk - 1);

    for (int i = threadIdx.x; i <= C; i += kMainThreads) pw[i] = exp2f(l2 * i);
    // powers that the tokens of a chunk have ahead of them: full chunks, and the short one
    for (int i = threadIdx.x; i < 2 * C; i += kMainThreads) {
        const int j = i % C, v = i < C ? C : vlast;
        wtab[i / C][j] = j < v ? exp2f(l2 * (rev ? j : v - 1 - j)) : 0.f;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_base;
    const int items = nchunk * reps;
    // scale gamma^n by which the state meets row i of chunk k (the first chunk of a reverse pass may be the short one and
    // has an offset; all others, and all of a forward pass, have the same)
    auto factor = [&](int k, int i) {
        const int valid = min(C, part.hi - chunk0(k));
        return row_factor(p.scale * pw[max((rev ? valid - i : i + 1) - (k == 0 ? off0 : 0), 0)]);
    };

    if (warp == 0) {
        // ---------------- TMA loads of x
        const CUtensorMap *mx = &maps.m[pi][0];
        const int tiles = many ? nchunk : items;
        Ring rx;
        int n = 0, k = 0, r = 0;   // n issued
#pragma unroll 1
        for (; n < tiles; ++n) {
            // (the first use of a stage: the phase before the first counts as over)
            if (!await(&x_empty[rx.s], rx.p ^ 1u, &abort_flag)) break;
            if (elect_one()) {
                uint8_t *x = xbuf + rx.s * K::X_BYTES;
                mbar_arrive_expect_tx(&x_full[rx.s], K::X_BYTES);
#pragma unroll
                for (int blk = 0; blk < DX / 64; ++blk)
                    tma_load_4d(x + blk * C * 128, mx, &x_full[rx.s], blk * 64, chunk0(k), many ? h : h * reps + r, b);
            }
            __syncwarp();
            rx.next(NX);
            if (many || ++r == reps) {
                r = 0;
                ++k;
            }
        }
        for (int i = n > NX ? n - NX : 0; i < n; ++i) warp_drain(&x_full[i % NX], (i / NX) & 1);
    } else if (warp == 3) {
        // ---------------- TMA loads of y and z
        const CUtensorMap *my = &maps.m[pi][1], *mz = &maps.m[pi][2];
        const int tiles = many ? items : nchunk;
        Ring ry, rz;
        int ny = 0, nz = 0, k = 0, r = 0;   // issued
#pragma unroll 1
        for (; ny < tiles; ++nz) {
            const int c0 = chunk0(k), hyz = many ? h * reps + r : h;
            if (!await(&y_empty[ry.s], ry.p ^ 1u, &abort_flag)) break;
            if (elect_one()) {
                uint8_t *y = ybuf + ry.s * K::Y_BYTES;
                mbar_arrive_expect_tx(&y_full[ry.s], K::Y_BYTES);
#pragma unroll
                for (int blk = 0; blk < DX / 64; ++blk)
                    tma_load_4d(y + blk * C * 128, my, &y_full[ry.s], blk * 64, c0, hyz, b);
            }
            __syncwarp();
            ry.next(NY);
            ++ny;
            if (!await(&z_empty[rz.s], rz.p ^ 1u, &abort_flag)) break;
            if (elect_one()) {
                uint8_t *z = zbuf + rz.s * K::Z_BYTES;
                mbar_arrive_expect_tx(&z_full[rz.s], K::Z_BYTES);
#pragma unroll
                for (int blk = 0; blk < DZ / 64; ++blk)
                    tma_load_4d(z + blk * C * 128, mz, &z_full[rz.s], blk * 64, c0, hyz, b);
            }
            __syncwarp();
            rz.next(NZ);
            if (!many || ++r == reps) {
                r = 0;
                ++k;
            }
        }
        for (int i = ny > NY ? ny - NY : 0; i < ny; ++i) warp_drain(&y_full[i % NY], (i / NY) & 1);
        for (int i = nz > NZ ? nz - NZ : 0; i < nz; ++i) warp_drain(&z_full[i % NZ], (i / NZ) & 1);
    } else if (warp == 1) {
        // ---------------- scores, and O = P Z (+ the decayed X times S_bf, once for each output tile).  With two
        // buffers the scores of the next item go ahead of this one's O where their tiles are in.  This warp's MMAs
        // run in the order of their issue, so scores cannot overtake the P and X that they replace
        constexpr uint32_t idA = idesc_bf16(128, C, false, false);
        constexpr uint32_t idO = idesc_bf16(128, DZ, false, true);
        const uint32_t tO = tm + K::T_O, sb = smem_u32(sbf), sl = smem_u32(slo);
        // of the next scores: x and y tile, buffer, item, chunk, head
        Ring sx, sy, sc;
        int si = 0, sk = 0, sr = 0;
        // of the item whose O is next: z tile, buffer, output tile (two barriers in turn, and one)
        Ring iz, ic, it2;
        uint32_t op = 1;
        int it = 0, k = 0, r = 0;
        // what can go next goes: the next item's scores when its tiles are in and a buffer is free, this item's O when
        // its P is made
        uint32_t idle = 0;
#pragma unroll 1
        while (it < items) {
            // (a tile with rows past the sequence's length, its last: those are zeroed first)
            const bool ragged = p.lengths && sk == nchunk - 1 && vlast < C;
            if (si < items && si < it + NSC && is_over(&x_full[sx.s], sx.p) && is_over(&y_full[sy.s], sy.p) &&
                (!ragged || is_over(&zeroed, 0))) {
                const bool last = sr == reps - 1;
                const uint32_t x = smem_u32(xbuf + sx.s * K::X_BYTES), y = smem_u32(ybuf + sy.s * K::Y_BYTES);
                tc_fence_after();
                LA_TL(si, 0);
                if (elect_one()) {
                    mma_ss_kk<DX / 16>(tm + K::T_A + sc.s * 128, desc_kmajor(x, C, 0, 0), desc_kmajor(y, C, 0, 0), idA);
                    mma_commit(&sc_full[sc.s]);
                    if (last || !many) mma_commit(&x_empty[sx.s]);
                    if (YSM && (last || many)) mma_commit(&y_scored[sy.s]);
                }
                __syncwarp();
                LA_TL(si, 1);
                if (last || !many) sx.next(NX);
                if (last || many) sy.next(NY);
                sc.next(NSC);
                ++si;
                if (++sr == reps) {
                    sr = 0;
                    ++sk;
                }
                idle = 0;
                continue;
            }
            if (si == it || !is_over(&p_ready[ic.s], ic.p)) {
                if (++idle > kTries) {
                    abort_flag = 1;
                    break;
                }
                continue;
            }
            idle = 0;
            const bool first = r == 0, last = r == reps - 1;
            const bool opens = first || !many, ends = last || !many;   // an output tile
            LA_TL(it, 4);
            const uint32_t z = smem_u32(zbuf + iz.s * K::Z_BYTES), tA = tm + K::T_A + ic.s * 128;
            if (opens) {
                // the state's part first: S moves on (in its own role) while P Z is under way
                if (!await(&o_free, op, &abort_flag)) break;   // (the first: the phase before it counts as over)
                if (!await(&xd_ready[it2.s], it2.p, &abort_flag)) break;
                if (first && !await(&s_conv, k & 1, &abort_flag)) break;
                LA_TL(it, 5);
                tc_fence_after();
                if (elect_one()) {
                    mma_ts_mn<DX / 16>(tO, tA + 64, desc_mnmajor(sl, DX, 0, 0), idO, 0u);
                    mma_ts_mn<DX / 16>(tO, tA + 64, desc_mnmajor(sb, DX, 0, 0), idO, 1u);
                    if (many ? first : last) mma_commit(&s_full);   // the chunk's last reader of S_hi, S_lo
                }
                __syncwarp();
            }
            if (!await(&z_full[iz.s], iz.p, &abort_flag)) break;
            LA_TL(it, 2);
            tc_fence_after();
            if (elect_one()) {
                mma_ts_mn<C / 16>(tO, tA, desc_mnmajor(z, C, 0, 0), idO, 1u);
                if (ends) mma_commit(&o_full);
                if (last || many) mma_commit(&z_empty[iz.s]);
            }
            __syncwarp();
            LA_TL(it, 6);
            if (ends) {
                it2.next(2);
                op ^= 1u;
            }
            if (last || many) iz.next(NZ);
            ic.next(NSC);
            ++it;
            if (++r == reps) {
                r = 0;
                ++k;
            }
        }
        if (elect_one()) mma_commit(&fin[0]);
        __syncwarp();
        warp_drain(&fin[0], 0);
    } else if (warp == 2) {
        // ---------------- S += Y^T Z, once for each y z tile
        constexpr uint32_t idS = idesc_bf16(128, DZ, YSM, true);
        const uint32_t tS = tm + K::T_S;
        const int tiles = many ? items : nchunk, per = many ? reps : 1;
        Ring ry, rz;
        int k = 0, r = 0;
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
            if (r == 0 && !await(&s_conv, k & 1, &abort_flag)) break;
            if (!await(&z_full[rz.s], rz.p, &abort_flag)) break;
            if (!await(&yt_ready[ry.s], ry.p, &abort_flag)) break;
            LA_TL(t, 3);
            tc_fence_after();
            const uint32_t y = smem_u32(ybuf + ry.s * K::Y_BYTES), z = smem_u32(zbuf + rz.s * K::Z_BYTES);
            const bool ends = ++r == per;
            if (elect_one()) {
                if constexpr (YSM) {
                    // (M = 128 rows d of which DX count: with 64 the others read what lies behind the tile)
                    mma_ss_mn8(tS, desc_mnmajor(y, C, 0, 0), desc_mnmajor(z, C, 0, 0), idS, 1u);
                    mma_commit(&y_empty[ry.s]);
                } else {
                    mma_ts_mn<C / 16>(tS, tm + K::T_Y, desc_mnmajor(z, C, 0, 0), idS, 1u);
                    mma_commit(&yt_done);
                }
                mma_commit(&z_empty[rz.s]);
                if (ends) mma_commit(&s_full);
                if constexpr (YSM) {   // the output goes where this z was, or not
                    if (o_in_z && ends)
                        mma_commit(&z_used[k % 2]);
                    else
                        mbar_arrive_cnt(&z_empty[rz.s], 4);
                }
            }
            __syncwarp();
            ry.next(NY);
            rz.next(NZ);
            if (ends) {
                r = 0;
                ++k;
            }
        }
        if (elect_one()) mma_commit(&fin[1]);
        __syncwarp();
        warp_drain(&fin[1], 0);
    } else if (warp >= 4 && warp < 8) {
        // ---------------- P = bf16(scale A o W / m), thread = row i, 32 columns at a time.  Away from the diagonal
        // gamma^|i - j| = gamma^(distance to the near end of a block of 16) gamma^(distance in the block); on it the blocks
        // of 16 have the lower (reverse: upper) triangle of one pattern, or are such a full block, or nothing.  Both
        // patterns stay in registers, with `scale`
        const int wq = warp % 4, lane = threadIdx.x % 32, i = wq * 32 + lane;
        float g[16], tri[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const int ago = rev ? e - lane % 16 : lane % 16 - e;
            g[e] = p.scale * pw[rev ? e : 15 - e];
            tri[e] = ago >= 0 ? p.scale * pw[max(ago, 0)] : 0.f;
        }
        const bool low = lane < 16;
        Ring sc, ry;
        int r = 0, ot = 0;
        float inv = __fdividef(1.f, factor(0, i).m);
#pragma unroll 1
        for (int it = 0; it < items; ++it) {
            if (!await(&sc_full[sc.s], sc.p, &abort_flag)) break;
            tc_fence_after();
            if (i == 127) LA_TL(it, 7);
            const uint32_t ta = tm + K::T_A + sc.s * 128 + ((uint32_t)(wq * 32) << 16);
            const bool first = r == 0, last = ++r == reps;
            if (it == reps && rev) inv = __fdividef(1.f, factor(1, i).m);
            if (!YSM && (last || many)) {
                mbar_arrive_w(&y_empty[ry.s]);
                ry.next(NY);
            }
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
                        const int near = rev ? j0 - i : i - j0 - 15;   // distance to the block's near end
                        const bool diag = cb == wq;
                        const float full = !diag || (rev ? hb == 1 && low : hb == 0 && !low) ? inv * pw[max(near, 0)] : 0.f;
                        const float half = diag && low == (hb == 0) ? inv : 0.f;
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            float a = g[e], b = g[e + 1];
                            mul2(a, b, full, full);
                            fma2(a, b, tri[e], tri[e + 1], half);
                            mul2(v[hb * 16 + e], v[hb * 16 + e + 1], a, b);
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
                }
                // over columns that this thread has read (16 cb .. 16 cb + 15 <= 32 cb + 31)
                tmem_st16_raw(ta + cb * 16, w);
            }
            tmem_st_wait();
            tc_fence_before();
            if (i == 127) LA_TL(it, 8);
#ifdef LA_TEST_HOOKS
            if (!(g_la_test_skip_decay == 1 && blockIdx.x == 0 && it == 0 && warp == 4))
#endif
                mbar_arrive_warp(&p_ready[sc.s]);
            sc.next(NSC);
            if (first || !many) mbar_arrive_warp(&p_first[ot++ & 1]);
            if (last) r = 0;
        }
    } else if (warp >= 8 && warp < 12) {
        // ---------------- S: the operands S_hi, S_lo of the state before the chunk, and its decay; thread = row d
        const int wq = warp % 4, d = wq * 32 + threadIdx.x % 32;
        const uint32_t ts = tm + K::T_S + ((uint32_t)(wq * 32) << 16);
        const bool have = wq * 32 < DX;
        const size_t E = (size_t)p.D * p.Dv;
        // element [d][e] of the pass's state is at d sd + e se of a state that the caller keeps
        const size_t sd = ps.tr ? 1 : p.Dv, se = ps.tr ? p.Dv : 1;
        // 32 columns of the segment's starting state
        auto start32 = [&](int e0, float *v) {
            if (p.nseg > 1) {
                const float4 *f = reinterpret_cast<const float4 *>(ps.slots + ((size_t)bg * p.nseg + u) * E + decay_blocked(DX, d, e0));
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float4 x = f[q * DX];
                    v[4 * q] = x.x;
                    v[4 * q + 1] = x.y;
                    v[4 * q + 2] = x.z;
                    v[4 * q + 3] = x.w;
                }
            } else if (ps.init) {
                const float *f = ps.init + (size_t)bg * E + d * sd + e0 * se;
                if (ps.tr) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = f[e * se];
                } else {
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const float4 x = reinterpret_cast<const float4 *>(f)[q];
                        v[4 * q] = x.x;
                        v[4 * q + 1] = x.y;
                        v[4 * q + 2] = x.z;
                        v[4 * q + 3] = x.w;
                    }
                }
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] *= ps.init_mul;
            } else {
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = 0.f;
            }
        };
        // the powers of gamma that S takes before each chunk's Y^T Z; first the chunk that starts from memory
        const float g0 = nchunk > 0 ? pw[min(C, part.hi - chunk0(0)) - off0] : 1.f;
        const float g = pw[C], gl = pw[rev ? C : vlast];
        if (have) {
#pragma unroll 1
            for (int c32 = 0; c32 < DZ / 32; ++c32) {
                float v[32];
                start32(c32 * 32, v);
                store_state_terms<DX>(sbf, slo, d, v, 2 * c32);
                store_state_terms<DX>(sbf, slo, d, v + 16, 2 * c32 + 1);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] *= g0;
                tmem_st16(ts + c32 * 32, v);
                tmem_st16(ts + c32 * 32 + 16, v + 16);
            }
            tmem_st_wait();
        }
#pragma unroll 1
        for (int k = 0; k < nchunk; ++k) {
            if (k > 0) {
                if (!await(&s_full, (k - 1) & 1, &abort_flag)) break;
                tc_fence_after();
                if (d == 0) LA_TL(k, 9);
                const float gk = k == nchunk - 1 ? gl : g;
                if (have) {
                    float va[16], vb[16];
                    auto part16 = [&](float *v, int c16) {
                        store_state_terms<DX>(sbf, slo, d, v, c16);
#pragma unroll
                        for (int e = 0; e < 16; e += 2) mul2(v[e], v[e + 1], gk, gk);
                        tmem_st16(ts + c16 * 16, v);
                    };
                    tmem_ld16(ts, va);
#pragma unroll 1
                    for (int c32 = 0; c32 < DZ / 32; ++c32) {
                        tmem_wait_regs<16>(va);
                        tmem_ld16(ts + c32 * 32 + 16, vb);
                        part16(va, 2 * c32);
                        tmem_wait_regs<16>(vb);
                        if (c32 + 1 < DZ / 32) tmem_ld16(ts + c32 * 32 + 32, va);
                        part16(vb, 2 * c32 + 1);
                    }
                    tmem_st_wait();
                }
            }
            fence_proxy_async();
            tc_fence_before();
            if (d == 0) LA_TL(k, 10);
            mbar_arrive_warp(&s_conv);
        }
    } else if (warp >= 12 && warp < 16) {
        // ---------------- the decayed X, thread = row i: made in registers while P is under way, stored where the
        // scores have been read.  2^e x, exact
        const int wq = warp % 4, i = wq * 32 + threadIdx.x % 32;
        const int tiles = many ? nchunk : items, step = many ? reps : 1;   // output tiles; items of each
        auto power = [&](int k) {
            const float g = factor(k, i).p2;
            return as_bf162(pack_bf16x2(g, g));
        };
        __nv_bfloat162 gh = power(0);
        Ring rx;
        int k = 0, r = 0;
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
            if (!await(&x_full[rx.s], rx.p, &abort_flag)) break;
            if (i == 0) LA_TL(t, 11);
            const uint8_t *x = xbuf + rx.s * K::X_BYTES;
            if (rev && k == 1) gh = power(1);
            uint32_t w[DX / 2];
#pragma unroll
            for (int c = 0; c < DX / 8; ++c) {
                const uint4 v = *reinterpret_cast<const uint4 *>(x + swz_chunk(C, i, c));
                const uint32_t a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) w[4 * c + e] = as_u32(__hmul2(as_bf162(a[e]), gh));
            }
            mbar_arrive_w(&x_empty[rx.s]);   // the tile is free for the next load
            rx.next(NX);
            if (!await(&p_first[t & 1], (t >> 1) & 1, &abort_flag)) break;
            tc_fence_after();
            const uint32_t tx = tm + K::T_A + ((t * step) % NSC) * 128 + 64 + ((uint32_t)(wq * 32) << 16);
#pragma unroll
            for (int q = 0; q < DX / 32; ++q) tmem_st16_raw(tx + q * 16, w + 16 * q);
            tmem_st_wait();
            tc_fence_before();
            if (i == 0) LA_TL(t, 12);
            mbar_arrive_warp(&xd_ready[t & 1]);
            if (many || ++r == reps) {
                r = 0;
                ++k;
            }
        }
    } else if (warp >= 16 && warp < 20) {
        // ---------------- the output rows, thread = row i; each warp stages and stores its own 32
        // (written from registers the rows, 32 bytes at a time, took a third of the chunk's time)
        const int wq = warp % 4, i = wq * 32 + threadIdx.x % 32;
        const uint32_t to = tm + K::T_O + ((uint32_t)(wq * 32) << 16);
        const int tiles = many ? nchunk : items;
        const CUtensorMap *mo = &maps.m[pi][3];
        float m = factor(0, i).m;
        int k = 0, r = 0;
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
            const int c0 = chunk0(k), valid = min(C, part.hi - c0), zi = o_in_z ? (many ? (t + 1) * reps - 1 : t) % NZ : 0;
            uint8_t *o = o_in_z ? zbuf + zi * K::Z_BYTES : obuf + (NO > 1 ? t % NO : 0) * K::O_BYTES;
            if (rev && k == 1) m = factor(1, i).m;
            if (!await(&o_full, t & 1, &abort_flag)) break;
            tc_fence_after();
            if (i == 0) LA_TL(t, 13);
            if (o_in_z && !await(&z_used[t & 1], (t >> 1) & 1, &abort_flag)) break;
            bulk_wait_read_but<(NO > 1 ? NO - 1 : 0)>();   // (of the elected lane)
            __syncwarp();
#pragma unroll 1
            for (int c32 = 0; c32 < DZ / 32; ++c32) {
                float v[32];
                tmem_ld32(to + c32 * 32, v);
                tmem_wait_regs<32>(v);
                if (c32 == DZ / 32 - 1) {   // O is free for the next item's products
                    tc_fence_before();
                    mbar_arrive_warp(&o_free);
                    if (i == 0) LA_TL(t, 14);
                }
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    mul2(v[2 * e], v[2 * e + 1], m, m);
                    w[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
                }
                if (i >= valid) {   // past the length: zeros
#pragma unroll
                    for (int e = 0; e < 16; ++e) w[e] = 0u;
                }
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<uint4 *>(o + swz_chunk(C, i, c32 * 4 + q)) =
                        make_uint4(w[4 * q], w[4 * q + 1], w[4 * q + 2], w[4 * q + 3]);
            }
            fence_proxy_async();
            __syncwarp();
            if (elect_one()) {
                if (c0 + wq * 32 < p.N)
#pragma unroll
                    for (int blk = 0; blk < DZ / 64; ++blk)
                        tma_store_4d(mo, o + blk * C * 128 + wq * 32 * 128, blk * 64, c0 + wq * 32, many ? h : h * reps + r, b);
                bulk_commit();
            }
            __syncwarp();
            if (o_in_z) {
                bulk_wait_read_but<0>();
                mbar_arrive_w(&z_empty[zi]);
            }
            if (many || ++r == reps) {
                r = 0;
                ++k;
            }
        }
        bulk_wait_all();
    } else if (warp >= 20) {
        // ---------------- the decayed y of every y z tile
        const int wq = warp % 4, j = threadIdx.x - 640;
        const uint32_t lane_off = (uint32_t)(wq * 32) << 16;
        const int tiles = many ? items : nchunk;
        YtWeights w;
        __nv_bfloat162 gh, gl;
        bool shorter = false;
        Ring ry, rz;
        int k = 0, r = 0;
#pragma unroll 1
        for (int t = 0; t < tiles; ++t) {
            const int c0 = chunk0(k), valid = min(C, part.hi - c0);
            uint8_t *y = ybuf + ry.s * K::Y_BYTES;
            if (!YSM || p.lengths)
                if (!await(&y_full[ry.s], ry.p, &abort_flag)) break;
            if (p.lengths) {
                if (!await(&z_full[rz.s], rz.p, &abort_flag)) break;
                if (valid < C) {
                    zero_rows<DX>(y, valid, j, 128);
                    zero_rows<DZ>(zbuf + rz.s * K::Z_BYTES, valid, j, 128);
                    fence_proxy_async();
                    mbar_arrive_warp(&zeroed);
                    // (the warps read one another's zeros)
                    if (!await(&zeroed, 0, &abort_flag)) break;
                }
            }
            const bool fresh = t == 0 || (valid < C) != shorter;
            shorter = valid < C;
            if constexpr (YSM) {
                // in place, thread = row (token) j, once the scores have read the tile
                if (fresh) {
                    const float g = wtab[shorter][j];
                    gh = as_bf162(pack_bf16x2(g, g));
                    const float gr = g - unpack_bf16x2(as_u32(gh)).x;
                    gl = as_bf162(pack_bf16x2(gr, gr));
                }
                if (!await(&y_scored[ry.s], ry.p, &abort_flag)) break;
#pragma unroll 4
                for (int c = 0; c < DX / 8; ++c) {
                    uint4 *q = reinterpret_cast<uint4 *>(y + swz_chunk(C, j, c));
                    uint4 v = *q;
                    v.x = as_u32(__hfma2(as_bf162(v.x), gh, __hmul2(as_bf162(v.x), gl)));
                    v.y = as_u32(__hfma2(as_bf162(v.y), gh, __hmul2(as_bf162(v.y), gl)));
                    v.z = as_u32(__hfma2(as_bf162(v.z), gh, __hmul2(as_bf162(v.z), gl)));
                    v.w = as_u32(__hfma2(as_bf162(v.w), gh, __hmul2(as_bf162(v.w), gl)));
                    *q = v;
                }
                fence_proxy_async();
            } else {
                if (fresh && wq * 32 < DX) w.set(wtab[shorter], 1.f);
                if (t > 0 && !await(&yt_done, (t - 1) & 1, &abort_flag)) break;
                tc_fence_after();
                if (wq * 32 < DX) {
                    yt_tile(y, wq * 32, w, tm + K::T_Y + lane_off);
                    tmem_st_wait();
                }
                mbar_arrive_w(&y_empty[ry.s]);
                tc_fence_before();
            }
            if (threadIdx.x == 640) LA_TL(t, 15);
            mbar_arrive_warp(&yt_ready[ry.s]);
            ry.next(NY);
            rz.next(NZ);
            if (!many || ++r == reps) {
                r = 0;
                ++k;
            }
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
// The sums over parts of segments (see DecayStateParams).  y is decayed to the part's end at once (y w, w <= 1).
//   Sums that only bf16 outputs depend on: bf16(y w)^T Z, in place of y, all in one accumulator.
//   A state that goes out: y w in float32 as three bf16 terms (all 24 bits), hi in place of y, mid and lo in tiles of
// their own.  The MMA's sums are cut, not rounded, to float32 at every step, so that long chains of them drift (2e-7 a
// chunk and head); each chunk and head has an accumulator of its own, smallest terms first, and eight warps add those up
// in registers.  1.3 to 3e-7 of the state, whatever its length (in two terms and one accumulator 4e-6 to 7e-5).
// Where a whole sequence is one part, these warps write the state itself (`direct`).
// Warps: 0 TMA, 1 MMA, 4-11 y (two threads a token), 12-19 the sums.  One term is bound by memory where the parts are long
// (8 heads, N 65536, 128 x 128: 58 us for 268 MB), else by the first chunk's latency (64 heads, N 4096, 64 x 64, parts of
// 8 chunks: 14 us).  Three terms take 69 us there, 73 us for 4 x 40 heads, N 4096, 128 x 64 (252 MB): the instructions that
// split y (without them 50 us; rounded instead of cut terms 85) and the terms' way through shared memory.
constexpr int kStateThreads = 640, kStateY = 256, kStateSum = 256;

struct StateMaps {
    CUtensorMap m[2][2];   // per array: y, z
};

template <int D, int DV>
struct StateCfg {
    static constexpr int Y_BYTES = C * D * 2, STAGE = Y_BYTES + C * DV * 2;
    // the MMA's M is 128 whatever D: what lies behind a y tile is its z tile, behind mid's tile lo's, and behind that one
    // there is room for the rest of 128 columns
    static constexpr int TERM_BYTES = Y_BYTES + C * 128 * 2;
    static constexpr int FIT = (kSmemLimit - 1024 - 2048 - TERM_BYTES) / STAGE, NS = FIT > 4 ? 4 : FIT;
    static constexpr int SMEM = NS * STAGE + TERM_BYTES + 1024;
    static_assert(D == 128 || STAGE - Y_BYTES >= C * 64 * 2, "128 columns from a y tile's start");
    static_assert(NS >= 2, "two stages");
    static constexpr int NA = 512 / DV;   // accumulators
};

template <int D, int DV>
__global__ void __launch_bounds__(kStateThreads, 1) k_decay_tc_state(const __grid_constant__ StateMaps maps,
                                                                     const __grid_constant__ DecayStateParams p) {
    using K = StateCfg<D, DV>;
    constexpr int NS = K::NS;
    extern __shared__ uint8_t smem_raw[];
    constexpr int NA = K::NA;
    __shared__ uint64_t full[NS], empty[NS], y_ready[NS], acc_full[NA], acc_empty[NA], terms_free, zeroed, fin;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    uint8_t *stage = align1024(smem_raw), *mid_tile = stage + NS * K::STAGE, *lo_tile = mid_tile + K::Y_BYTES;
    pdl_wait();
    const int warp = threadIdx.x / 32;
    // the block's parts, one after the other (no wave of blocks starts anew); every role walks them.  The last in token
    // order, which may be short, come last
    const int nparts = p.nsum * p.nsub, total = p.n * nparts * p.B * p.Hkv;
    struct Task {
        int a, bg, b, h, pidx, lo, hi, rev, heads, nchunk, items;
        bool exact;
        float l2;
        // chunks in the pass's order, the smallest powers first (small terms after large ones would be cut at their size)
        __device__ __forceinline__ int chunk0(int it) const {
            return lo + C * (rev ? nchunk - 1 - it / heads : it / heads);
        }
    };
    auto task = [&](int i) {
        Task t;
        const int ah = i % (p.n * p.B * p.Hkv), q = i / (p.n * p.B * p.Hkv);
        t.a = p.first + ah / (p.B * p.Hkv);
        t.pidx = p.rev[t.a] ? nparts - 1 - q : q;
        t.bg = ah % (p.B * p.Hkv);
        t.b = t.bg / p.Hkv;
        t.h = t.bg % p.Hkv;
        t.rev = p.rev[t.a];
        t.heads = p.heads[t.a];
        t.exact = p.exact[t.a];
        const Part part = sub_part_of(decay_tokens(p.lengths, t.b, p.N), p.N, t.pidx / p.nsub, p.nseg, p.seg_len,
                                      t.pidx % p.nsub, p.nsub, p.sub_len, t.rev);
        t.lo = part.lo;
        t.hi = part.hi;
        t.nchunk = (part.hi - part.lo + C - 1) / C;
        t.items = t.nchunk * t.heads;
        t.l2 = decay_log2(p.log_decay[t.h]);
        return t;
    };
    if (threadIdx.x == 0) {
        abort_flag = 0;
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
            mbar_init(&y_ready[s], kStateY);
        }
        for (int s = 0; s < NA; ++s) {
            mbar_init(&acc_full[s], 1);
            mbar_init(&acc_empty[s], kStateSum);
        }
        mbar_init(&terms_free, 1);
        mbar_init(&zeroed, kStateY);
        mbar_init(&fin, 1);
        fence_barrier_init();
    }
    if (threadIdx.x >= 96 && threadIdx.x < 98) tma_prefetch_map(&maps.m[p.first][threadIdx.x - 96]);
    if (warp == 1) {
        tmem_alloc(&tmem_base, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = tmem_base;
    bool ok = true;
    if (warp == 0) {
        Ring st;
        int issued = 0;
        for (int i = blockIdx.x; ok && i < total; i += gridDim.x) {
            const Task t = task(i);
            for (int it = 0; it < t.items; ++it) {
                const int c0 = t.chunk0(it), hh = t.h * t.heads + it % t.heads;
                // (the first use of a stage: the phase before the first counts as over)
                if (!(ok = await(&empty[st.s], st.p ^ 1u, &abort_flag))) break;
                uint8_t *y = stage + st.s * K::STAGE, *z = y + K::Y_BYTES;
                if (elect_one()) {
                    const CUtensorMap *m = maps.m[t.a];
                    mbar_arrive_expect_tx(&full[st.s], K::STAGE);
#pragma unroll
                    for (int blk = 0; blk < D / 64; ++blk) tma_load_4d(y + blk * C * 128, &m[0], &full[st.s], blk * 64, c0, hh, t.b);
#pragma unroll
                    for (int blk = 0; blk < DV / 64; ++blk) tma_load_4d(z + blk * C * 128, &m[1], &full[st.s], blk * 64, c0, hh, t.b);
                }
                __syncwarp();
                st.next(NS);
                ++issued;
            }
        }
        for (int i = issued > NS ? issued - NS : 0; i < issued; ++i) warp_drain(&full[i % NS], (i / NS) & 1);
    } else if (warp == 1) {
        constexpr uint32_t id = idesc_bf16(128, DV, true, true);
        // (M = 128 rows d of which D count: with 64 the others read what lies behind the tile)
        Ring st, ac;
        for (int i = blockIdx.x; ok && i < total; i += gridDim.x) {
            const Task t = task(i);
            for (int it = 0; it < t.items; ++it) {
                const bool opens = t.exact || it == 0, ends = t.exact || it == t.items - 1;   // an accumulator
                if (opens && !(ok = await(&acc_empty[ac.s], ac.p ^ 1u, &abort_flag))) break;
                if (!(ok = await(&y_ready[st.s], st.p, &abort_flag))) break;
                tc_fence_after();
                const uint32_t y = smem_u32(stage + st.s * K::STAGE), z = y + K::Y_BYTES, acc = tm + ac.s * DV;
                if (elect_one()) {
                    if (t.exact) {
                        mma_ss_mn8(acc, desc_mnmajor(smem_u32(lo_tile), C, 0, 0), desc_mnmajor(z, C, 0, 0), id, 0u);
                        mma_ss_mn8(acc, desc_mnmajor(smem_u32(mid_tile), C, 0, 0), desc_mnmajor(z, C, 0, 0), id, 1u);
                        mma_commit(&terms_free);
                    }
                    mma_ss_mn8(acc, desc_mnmajor(y, C, 0, 0), desc_mnmajor(z, C, 0, 0), id, t.exact || it > 0 ? 1u : 0u);
                    mma_commit(&empty[st.s]);
                    if (ends) mma_commit(&acc_full[ac.s]);
                }
                __syncwarp();
                st.next(NS);
                if (ends) ac.next(NA);
            }
        }
        if (elect_one()) mma_commit(&fin);
        __syncwarp();
        warp_drain(&fin, 0);
    } else if (warp >= 4 && warp < 12) {
        const int thr = threadIdx.x - 128, j = thr % C, half = thr / C;
        Ring st;
        uint32_t free_p = 1, zero_p = 0;   // (the first use of the terms' tiles: the phase before it counts as over)
        for (int i = blockIdx.x; ok && i < total; i += gridDim.x) {
            const Task t = task(i);
            for (int it = 0; it < t.items; ++it) {
                const int c0 = t.chunk0(it), valid = min(C, t.hi - c0);
                if (!(ok = await(&full[st.s], st.p, &abort_flag))) break;
                uint8_t *y = stage + st.s * K::STAGE;
                if (p.lengths && valid < C) {
                    zero_rows<D>(y, valid, thr, kStateY);
                    zero_rows<DV>(y + K::Y_BYTES, valid, thr, kStateY);
                    mbar_arrive_warp(&zeroed);
                    if (!(ok = await(&zeroed, zero_p, &abort_flag))) break;
                    zero_p ^= 1u;
                }
                // what token j has ahead of it in the part
                const float g = exp2f(t.l2 * max(t.rev ? c0 + j - t.lo : t.hi - 1 - c0 - j, 0));
                if (t.exact) {
                    // (the terms are found beside the MMAs of the item before)
                    uint32_t m[D / 16][4], l[D / 16][4];
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        uint4 *q = reinterpret_cast<uint4 *>(y + swz_chunk(C, j, half * (D / 16) + c));
                        const uint4 v = *q;
                        const uint32_t x[4] = {v.x, v.y, v.z, v.w};
                        uint32_t h[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float2 f = unpack_bf16x2(x[e]);
                            mul2(f.x, f.y, g, g);
                            h[e] = cut_bf16x2(f);
                            m[c][e] = cut_bf16x2(f);
                            l[c][e] = cut_bf16x2(f);
                        }
                        *q = make_uint4(h[0], h[1], h[2], h[3]);
                    }
                    if (!(ok = await(&terms_free, free_p, &abort_flag))) break;
                    free_p ^= 1u;
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        const uint32_t at = swz_chunk(C, j, half * (D / 16) + c);
                        *reinterpret_cast<uint4 *>(mid_tile + at) = make_uint4(m[c][0], m[c][1], m[c][2], m[c][3]);
                        *reinterpret_cast<uint4 *>(lo_tile + at) = make_uint4(l[c][0], l[c][1], l[c][2], l[c][3]);
                    }
                } else {
                    const __nv_bfloat162 gh = as_bf162(pack_bf16x2(g, g));
                    const float gr = g - unpack_bf16x2(as_u32(gh)).x;
                    const __nv_bfloat162 gl = as_bf162(pack_bf16x2(gr, gr));
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        uint4 *q = reinterpret_cast<uint4 *>(y + swz_chunk(C, j, half * (D / 16) + c));
                        uint4 v = *q;
                        v.x = as_u32(__hfma2(as_bf162(v.x), gh, __hmul2(as_bf162(v.x), gl)));
                        v.y = as_u32(__hfma2(as_bf162(v.y), gh, __hmul2(as_bf162(v.y), gl)));
                        v.z = as_u32(__hfma2(as_bf162(v.z), gh, __hmul2(as_bf162(v.z), gl)));
                        v.w = as_u32(__hfma2(as_bf162(v.w), gh, __hmul2(as_bf162(v.w), gl)));
                        *q = v;
                    }
                }
                fence_proxy_async();
#ifdef LA_TEST_HOOKS
                if (!(g_la_test_skip_decay == 2 && i == 0 && it == 0 && warp == 4))
#endif
                    mbar_arrive_warp(&y_ready[st.s]);
                st.next(NS);
            }
        }
    } else if (warp >= 12) {
        // thread = row d, half of the columns
        constexpr int H = DV / 2;
        const int wq = warp % 4, d = wq * 32 + threadIdx.x % 32, e0 = (warp - 12) / 4 * H;
        const uint32_t ta = tm + ((uint32_t)(wq * 32) << 16) + e0;
        const bool have = wq * 32 < D;
        Ring ac;
        for (int i = blockIdx.x; i < total; i += gridDim.x) {
            const Task t = task(i);
            const int sums = t.exact ? t.items : min(t.items, 1);
            float S[H];
#pragma unroll
            for (int e = 0; e < H; ++e) S[e] = 0.f;
            for (int it = 0; it < sums; ++it) {
                if (!(ok = await(&acc_full[ac.s], ac.p, &abort_flag))) break;
                tc_fence_after();
                if (have) {
#pragma unroll
                    for (int c16 = 0; c16 < H / 16; ++c16) {
                        float v[16];
                        tmem_ld16(ta + ac.s * DV + c16 * 16, v);
                        tmem_wait_regs<16>(v);
#pragma unroll
                        for (int e = 0; e < 16; ++e) S[c16 * 16 + e] += v[e];
                    }
                }
                tc_fence_before();
                mbar_arrive_warp(&acc_empty[ac.s]);
                ac.next(NA);
            }
            if (!ok) break;
            if (have && p.direct) {
                // the state after the last token (what leaves a reverse pass decays once more)
                const int len = t.hi - t.lo, off = p.first_off[t.a];
                const float g = p.init_mul[t.a] * exp2f(t.l2 * max(len - off, 0));
                const float m = p.fin_mul[t.a] * (off && len > 0 ? exp2f(t.l2 * off) : 1.f);
                const size_t at = ((size_t)t.bg * D + d) * DV + e0;
#pragma unroll
                for (int e = 0; e < H; e += 4) {
                    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (p.init[t.a]) x = *reinterpret_cast<const float4 *>(p.init[t.a] + at + e);
                    *reinterpret_cast<float4 *>(p.fin[t.a] + at + e) =
                        make_float4(m * fmaf(g, x.x, S[e]), m * fmaf(g, x.y, S[e + 1]), m * fmaf(g, x.z, S[e + 2]),
                                    m * fmaf(g, x.w, S[e + 3]));
                }
            } else if (have) {
                float4 *f = reinterpret_cast<float4 *>(p.part[t.a] + ((size_t)t.bg * nparts + t.pidx) * D * DV + decay_blocked(D, d, e0));
#pragma unroll
                for (int e = 0; e < H / 4; ++e) f[e * D] = make_float4(S[4 * e], S[4 * e + 1], S[4 * e + 2], S[4 * e + 3]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_dealloc(tm, 512);
    if (threadIdx.x == 0 && abort_flag) atomicExch(p.err, kErrTimeout);
}

// ---------------------------------------------------------------------------------------
// Starting states of the segments, and the last state where it is an output: T = the given state, then for each
// segment (or part) T = gamma^tokens T + its sum, a thread carrying 4 x 4 elements; all states lane-blocked but the caller's.
// A few microseconds of latency (4 to 9; eight parts loaded ahead instead of four do not shorten them).  Lane-blocked,
// as a thread of the passes reads a whole row: from plain [D][Dv] states that took up to 50 us.
constexpr int kJoinThreads = 64;

template <int D, int DV>
__global__ void __launch_bounds__(kJoinThreads) k_decay_join(const __grid_constant__ DecayStateParams p) {
    pdl_wait();
    constexpr int kBlocks = D * DV / 16 / kJoinThreads;   // of one state
    const int ah = blockIdx.x / kBlocks, a = p.first + ah / (p.B * p.Hkv), bg = ah % (p.B * p.Hkv), b = bg / p.Hkv, h = bg % p.Hkv;
    const int idx = blockIdx.x % kBlocks * kJoinThreads + threadIdx.x, d = idx % (D / 4) * 4, e = idx / (D / 4) * 4;
    constexpr size_t E = (size_t)D * DV;
    const int n = decay_tokens(p.lengths, b, p.N), nparts = p.nsum * p.nsub;
    const float l2 = decay_log2(p.log_decay[h]);
    float4 t[4];   // rows d .. d + 3, columns e .. e + 3
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        t[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (p.init[a]) {
            const float4 x = *reinterpret_cast<const float4 *>(p.init[a] + bg * E + (size_t)(d + i) * DV + e);
            const float m = p.init_mul[a];
            t[i] = make_float4(x.x * m, x.y * m, x.z * m, x.w * m);
        }
    }
    const float4 *src = reinterpret_cast<const float4 *>(p.part[a] + (size_t)bg * nparts * E + decay_blocked(D, d, e));
    auto store = [&](int u) {
        if (p.start[a]) {
            float4 *o = reinterpret_cast<float4 *>(p.start[a] + ((size_t)bg * p.nseg + u) * E + decay_blocked(D, d, e));
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = t[i];
        }
        if (p.start_tr[a]) {
            float4 *o = reinterpret_cast<float4 *>(p.start_tr[a] + ((size_t)bg * p.nseg + u) * E + decay_blocked(DV, e, d));
            o[0] = make_float4(t[0].x, t[1].x, t[2].x, t[3].x);
            o[1] = make_float4(t[0].y, t[1].y, t[2].y, t[3].y);
            o[2] = make_float4(t[0].z, t[1].z, t[2].z, t[3].z);
            o[3] = make_float4(t[0].w, t[1].w, t[2].w, t[3].w);
        }
    };
    // the last state where it is an output: each part straight to the end (the same rounding of gamma^tokens from part to
    // part would add up: 1.3e-6 over 32 of them, 2e-7 so)
    float4 f[4];
    {
        const float g = exp2f(l2 * max(n - p.first_off[a], 0));
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = make_float4(g * t[i].x, g * t[i].y, g * t[i].z, g * t[i].w);
    }
    store(0);
    int off = p.first_off[a];
    // kAhead parts' sums are on their way at a time: one after the other costs a memory latency each
    constexpr int kAhead = 4;
    for (int i0 = 0; i0 < nparts; i0 += kAhead) {
        float4 x[kAhead][4];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[j][i] = i0 + j < nparts ? src[(size_t)(i0 + j) * (E / 4) + i] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (i0 + j >= nparts) break;
            const int u = (i0 + j) / p.nsub, s = (i0 + j) % p.nsub;
            const Part part = sub_part_of(n, p.N, u, p.nseg, p.seg_len, s, p.nsub, p.sub_len, p.rev[a]);
            const int len = part.hi - part.lo;
            const float g = exp2f(l2 * max(len - off, 0));
            if (len > 0) off = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i)
                t[i] = make_float4(fmaf(g, t[i].x, x[j][i].x), fmaf(g, t[i].y, x[j][i].y), fmaf(g, t[i].z, x[j][i].z),
                                   fmaf(g, t[i].w, x[j][i].w));
            if (p.fin[a]) {
                const float gf = exp2f(l2 * (p.rev[a] ? part.lo : n - part.hi));
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    f[i] = make_float4(fmaf(gf, x[j][i].x, f[i].x), fmaf(gf, x[j][i].y, f[i].y), fmaf(gf, x[j][i].z, f[i].z),
                                       fmaf(gf, x[j][i].w, f[i].w));
            }
            if (s == p.nsub - 1 && u + 1 < p.nseg) store(u + 1);
        }
    }
    if (p.fin[a]) {
        // all segments summed: the state after the last token (what leaves a reverse pass decays once more)
        const float m = p.fin_mul[a] * (p.first_off[a] && n > 0 ? exp2f(l2 * p.first_off[a]) : 1.f);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            *reinterpret_cast<float4 *>(p.fin[a] + bg * E + (size_t)(d + i) * DV + e) =
                make_float4(f[i].x * m, f[i].y * m, f[i].z * m, f[i].w * m);
    }
}

// ---- launches ---------------------------------------------------------------------------

template <int DX, int DZ>
cudaError_t passes_d(const DecayParams &p, int pass0, int npass, cudaStream_t s) {
    PassMaps maps;
    for (int i = pass0; i < pass0 + npass; ++i) {
        const DecayPass &ps = p.pass[i];
        const int Hq = p.Hkv * p.n_rep, Hx = ps.many_yz ? p.Hkv : Hq, Hyz = ps.many_yz ? Hq : p.Hkv;
        cudaError_t e = make_map_in(&maps.m[i][0], ps.x, p.B, Hx, p.N, DX, ps.sx, C);
        if (e == cudaSuccess) e = make_map_in(&maps.m[i][1], ps.y, p.B, Hyz, p.N, DX, ps.sy, C);
        if (e == cudaSuccess) e = make_map_in(&maps.m[i][2], ps.z, p.B, Hyz, p.N, DZ, ps.sz, C);
        if (e == cudaSuccess) e = make_map_in(&maps.m[i][3], ps.out, p.B, Hx, p.N, DZ, contiguous_strides(Hx, p.N, DZ), 32);
        if (e != cudaSuccess) return e;
    }
    auto kern = k_decay_tc<DX, DZ>;
    constexpr int smem = MainCfg<DX, DZ>::SMEM;
    cudaError_t e = prepare(kern, smem);
    if (e != cudaSuccess) return e;
    TraceScope tr("decay_tc", s);
    return launch_pdl(kern, dim3((unsigned)npass * p.nseg * p.B * p.Hkv), dim3(kMainThreads), smem, s, maps, p, pass0, npass);
}

cudaError_t passes(const DecayParams &p, int pass0, int npass, cudaStream_t s) {
    const bool tr = p.pass[pass0].tr;
    const int DX = tr ? p.Dv : p.D, DZ = tr ? p.D : p.Dv;
    if (DZ == 64) return DX == 64 ? passes_d<64, 64>(p, pass0, npass, s) : passes_d<128, 64>(p, pass0, npass, s);
    return DX == 64 ? passes_d<64, 128>(p, pass0, npass, s) : passes_d<128, 128>(p, pass0, npass, s);
}

template <int D, int DV>
cudaError_t states_d(const DecayStateParams &p, cudaStream_t s) {
    StateMaps maps;
    for (int a = p.first; a < p.first + p.n; ++a) {
        cudaError_t e = make_map_in(&maps.m[a][0], p.y[a], p.B, p.Hkv * p.heads[a], p.N, D, p.sy[a], C);
        if (e == cudaSuccess) e = make_map_in(&maps.m[a][1], p.z[a], p.B, p.Hkv * p.heads[a], p.N, DV, p.sz[a], C);
        if (e != cudaSuccess) return e;
    }
    auto kern = k_decay_tc_state<D, DV>;
    cudaError_t e = prepare(kern, StateCfg<D, DV>::SMEM);
    if (e != cudaSuccess) return e;
    TraceScope tr("decay_tc_state", s);
    const long long total = (long long)p.n * p.nsum * p.nsub * p.B * p.Hkv;
    return launch_pdl(kern, dim3(total < kPlanSms ? (unsigned)total : kPlanSms), dim3(kStateThreads), StateCfg<D, DV>::SMEM, s,
                      maps, p);
}

}  // namespace

cudaError_t decay_tc_states(const DecayStateParams &p, cudaStream_t s) {
    if (p.D == 64) return p.Dv == 64 ? states_d<64, 64>(p, s) : states_d<64, 128>(p, s);
    return p.Dv == 64 ? states_d<128, 64>(p, s) : states_d<128, 128>(p, s);
}

cudaError_t decay_tc_join(const DecayStateParams &p, cudaStream_t s) {
    auto kern = p.D == 64 ? (p.Dv == 64 ? k_decay_join<64, 64> : k_decay_join<64, 128>)
                          : (p.Dv == 64 ? k_decay_join<128, 64> : k_decay_join<128, 128>);
    TraceScope tr("decay_join", s);
    return launch_pdl(kern, dim3(p.D * p.Dv / 16 / kJoinThreads * (unsigned)(p.n * p.B * p.Hkv)), dim3(kJoinThreads), 0, s, p);
}

cudaError_t decay_tc_passes(const DecayParams &p, cudaStream_t s) {
    // the gradients' passes have two shapes of state, D x Dv and its transpose
    if (p.npass == 1 || p.D == p.Dv) return passes(p, 0, p.npass, s);
    cudaError_t e = passes(p, 0, 2, s);
    return e == cudaSuccess ? passes(p, 2, 1, s) : e;
}

}  // namespace la

#ifdef LA_TEST_HOOKS
// Test builds only: arm the withheld arrival of the passes (1) or of the sums (2), or disarm it (0).
extern "C" int la_test_withhold_decay(int which) {
    return cudaMemcpyToSymbol(la::g_la_test_skip_decay, &which, sizeof(int)) == cudaSuccess ? 0 : 1;
}
#endif

#ifdef LA_TIMELINE
extern "C" int la_timeline_read_decay(long long *out) {
    return cudaMemcpyFromSymbol(out, la::g_la_tl, sizeof(long long) * 64 * 16) == cudaSuccess ? 0 : 1;
}
#endif
