// la_ssm.cuh -- selective state space scan: launch parameters, work plan and the device functions that the scan, its
// gradient and its single-token step share.
//
//   d = softplus(dt + dt_bias)           (or dt + dt_bias)
//   h <- exp(d A) h + d x B,   y = C . h + skip x,   out = y z sigmoid(z)
//
// Every channel has S states of its own; B and C rows are shared by the channels of a group.
#pragma once

#include "la_internal.cuh"

namespace la {

constexpr int kSsmTile = 8;   // tokens between the states that the forward keeps for the gradient

// Strides of a [B, N, E] input (h unused), or of a [B, N, G, S] one (h: along G).
struct SsmParams {
    const void *x, *dt, *B, *C, *z, *g;
    Strides sx, sdt, sB, sC, sz, sg;
    const float *A, *skip, *dt_bias, *init, *dfinal;
    const int *lengths;
    void *out;                       // scan; NULL: only the kept states (and the final one) are wanted
    float *fin;                      // final state or NULL
    float *kept;                     // states at every kSsmTile tokens [B][tiles][S / 4][E][4] (written by the scan, read by the gradient)
    void *dx, *ddt, *dz;
    float *dinit;
    int nB, N, E, S, G, Eg, softplus;
    int seg_len, nseg;               // the launch's work split (a multiple of the kernels' tiles)
    float *seg_state;                // [B][nseg][E][S] sums of the segments alone
    float *seg_d;                    // [B][nseg][E] their sums of d
    float *part_bc;                  // gradient: [G * blocks][B][N][2 S] dB and dC summed over a block's channels
    float *part_A;                   // [B * nseg][E][S]
    float *part_e;                   // [B * nseg][2][E]: skip's and dt_bias' gradients
};

// What reduces the gradient's parts.
struct SsmReduceParams {
    const float *part_bc, *part_A, *part_e;
    const int *lengths;
    void *dB, *dC;
    float *dA, *dskip, *dbias;
    int nB, N, E, S, G, blocks, parts;   // blocks of a group's channels; parts: B * nseg
};

struct SsmStepParams {
    const void *x, *dt, *B, *C, *z;
    Strides sx, sdt, sB, sC, sz;
    const float *A, *skip, *dt_bias, *state;
    float *state_out;
    const int *slots;
    void *out;
    int pool, nB, E, S, G, Eg, softplus;
};

cudaError_t ssm_scan(const SsmParams &p, la_dtype dt, cudaStream_t s);             // p.nseg > 1: after ssm_segments
cudaError_t ssm_segments(const SsmParams &p, la_dtype dt, bool reverse, cudaStream_t s);
cudaError_t ssm_grad(const SsmParams &p, la_dtype dt, cudaStream_t s);
cudaError_t ssm_reduce(const SsmReduceParams &p, la_dtype dt, cudaStream_t s);
cudaError_t ssm_step(const SsmStepParams &p, la_dtype dt, cudaStream_t s);
int ssm_scan_channels(int S);    // channels of a block of the scan
int ssm_grad_channels(int S);    // ... and of the gradient

#ifdef __CUDACC__

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float ex2(float x) {   // 2^x: 1.4e-7 relative, 32 a clock and SM on GB300
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Two floats in one register pair: one instruction for two products or sums.
struct F2 {
    float x, y;
};
__device__ __forceinline__ F2 f2(float a) { return F2{a, a}; }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("{\n.reg .b64 a, b, c;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmov.b64 c, {%6, %7};\n"
        "fma.rn.f32x2 a, a, b, c;\nmov.b64 {%0, %1}, a;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("{\n.reg .b64 a, b;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nmul.rn.f32x2 a, a, b;\nmov.b64 {%0, %1}, a;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("{\n.reg .b64 a, b;\nmov.b64 a, {%2, %3};\nmov.b64 b, {%4, %5};\nadd.rn.f32x2 a, a, b;\nmov.b64 {%0, %1}, a;\n}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
// Decays 2^(d A) (A times log2(e)).  The instruction errs towards zero on average, and a decay's error adds up over all that a
// state remembers, so the exponent is raised first (an fma in place of the product).  What is on average right differs by the
// exponent: it errs by -5e-9 to -8e-9 for |x| in 1e-5 .. 2^-8, by -1.7e-8 to -2.5e-8 in 2^-8 .. 1.  A lane of the scan takes the
// one or the other for eight tokens, by what its slowest state, which remembers the most, meets at the first of them (so that no
// token has a part in the rows before it).  That leaves 2e-9 below 2^-8 and 6e-9 above it, and up to 2e-8, still less than
// without, for the faster states of a lane whose slowest one is below.  65536 x 2048 x 16: 973 us with one constant, 990 so.
// (2^tilt is 1 for either: a step of 0 changes nothing.)
constexpr float kTiltSlow = 9e-9f, kTilt = 2.8e-8f;
__device__ __forceinline__ F2 tilt_of(float x) { return f2(fabsf(x) < 0x1p-8f ? kTiltSlow : kTilt); }
__device__ __forceinline__ F2 decay2(F2 d, F2 A, F2 tilt) {
    const F2 x = fma2(d, A, tilt);
    return F2{ex2(x.x), ex2(x.y)};
}
// 2^(d A) h + sum for a whole segment, whose steps add up to d.  Its factor alone may be past 2^128 (A > 0) where the result is
// not, so its root is applied twice.  The root is at most 2^127.9, for a state of 0 has to stay 0; twice that takes any
// normal state past 2^128.  (min.NaN: a NaN in d stays one.)
__device__ __forceinline__ float join(float d, float A, float h, float sum) {
    float x = 0.5f * fmaf(d, A, kTilt);
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(x), "f"(127.9f));
    const float root = ex2(x);
    return fmaf(root, root * h, sum);
}

// log(1 + e) / e on [0, 1]: near the polynomial of its degree with the least relative error (5e-9, by Lawson's reweighted least
// squares); with coefficients rounded to float32 it errs by 3.8e-8, in float32 arithmetic by 1.2e-7.  No cancellation for small e,
// where log(1 + e) itself loses what 1 + e rounds away.
__device__ __forceinline__ float log1p_over(float e) {
    float a = -0.003243980696424842f;
    a = fmaf(a, e, 0.019851261749863625f);
    a = fmaf(a, e, -0.056959159672260284f);
    a = fmaf(a, e, 0.10603617131710052f);
    a = fmaf(a, e, -0.15305569767951965f);
    a = fmaf(a, e, 0.19675931334495544f);
    a = fmaf(a, e, -0.24954132735729218f);
    a = fmaf(a, e, 0.3332996368408203f);
    a = fmaf(a, e, -0.4999990165233612f);
    return fmaf(a, e, 1.0f);
}
__device__ __forceinline__ F2 log1p_over(F2 e) {
    F2 a = f2(-0.003243980696424842f);
    a = fma2(a, e, f2(0.019851261749863625f));
    a = fma2(a, e, f2(-0.056959159672260284f));
    a = fma2(a, e, f2(0.10603617131710052f));
    a = fma2(a, e, f2(-0.15305569767951965f));
    a = fma2(a, e, f2(0.19675931334495544f));
    a = fma2(a, e, f2(-0.24954132735729218f));
    a = fma2(a, e, f2(0.3332996368408203f));
    a = fma2(a, e, f2(-0.4999990165233612f));
    return fma2(a, e, f2(1.0f));
}
// softplus(v) = max(v, 0) + log(1 + exp(-|v|)); e = exp(-|v|) for its derivative.
__device__ __forceinline__ float softplus(float v, float &e) {
    e = ex2(-fabsf(v) * kLog2e);
    return fmaf(e, log1p_over(e), fmaxf(v, 0.f));
}
__device__ __forceinline__ F2 softplus(F2 v, F2 &e) {
    e = F2{ex2(-fabsf(v.x) * kLog2e), ex2(-fabsf(v.y) * kLog2e)};
    return fma2(e, log1p_over(e), F2{fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)});
}
__device__ __forceinline__ float sigmoid(float z) { return rcp(1.f + ex2(-z * kLog2e)); }
__device__ __forceinline__ F2 sigmoid(F2 z) {
    const F2 e = mul2(z, f2(-kLog2e)), s = add2(F2{ex2(e.x), ex2(e.y)}, f2(1.f));
    return F2{rcp(s.x), rcp(s.y)};
}

// A warp's lanes: channel lane % CPW, part r = lane / CPW of its states (CPW = 32 / LPC): lanes of the same part are neighbours,
// which makes their common loads of B and C 2 cycles of shared memory each instead of 4.
//
// Sums of v[j], of NT tokens each, over the LPC lanes of a channel, each sum left with the lane that owns token j: lane
// part r owns tokens r OWN .. r OWN + OWN - 1 (OWN = NT / LPC; with more lanes than tokens, parts r and r + NT own token r).
// Halves are exchanged, so that 8 sums over 4 lanes take 6 shuffles instead of 16.
template <int LPC, int NT>
__device__ __forceinline__ void part_sums(float (&v)[NT], int lane) {
    constexpr int CPW = 32 / LPC;
    int n = NT;
#pragma unroll
    for (int m = LPC / 2; m >= NT && m >= 1; m >>= 1)
#pragma unroll
        for (int i = 0; i < NT; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], m * CPW);
#pragma unroll
    for (int m = (LPC < NT ? LPC : NT) / 2; m >= 1; m >>= 1) {
        n >>= 1;
        const bool up = lane & (m * CPW);
#pragma unroll
        for (int i = 0; i < NT / 2; ++i)
            if (i < n) {
                const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m * CPW);
            }
    }
}

__device__ __forceinline__ void copy_async(void *dst, const void *src, bool there) {   // 16 bytes, zeros where not there
    const unsigned d = (unsigned)__cvta_generic_to_shared(dst);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(d), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Eight elements (16 or 32 bytes) as float32 to shared memory.
__device__ __forceinline__ void widen16(float *dst, const __nv_bfloat16 *src) {
    const uint4 v = *reinterpret_cast<const uint4 *>(src);
    auto lo = [](unsigned w) { return __uint_as_float(w << 16); };
    auto hi = [](unsigned w) { return __uint_as_float(w & 0xffff0000u); };
    *reinterpret_cast<float4 *>(dst) = make_float4(lo(v.x), hi(v.x), lo(v.y), hi(v.y));
    *reinterpret_cast<float4 *>(dst + 4) = make_float4(lo(v.z), hi(v.z), lo(v.w), hi(v.w));
}
__device__ __forceinline__ void widen16(float *dst, const float *src) {
    *reinterpret_cast<float4 *>(dst) = *reinterpret_cast<const float4 *>(src);
}

#endif

}  // namespace la
