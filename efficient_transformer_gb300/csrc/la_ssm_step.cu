// la_ssm_step.cu -- selective state space scan, one token of each sequence on a pool of states.
//
//   h <- exp(d A) h + d x B,   out = (C . h + skip x) z sigmoid(z)
//
// Bound by memory: a state is read and written once for 4 operations and an ex2.  A thread holds 4 states of one channel for
// each of U sequences (a 16-byte load each; A, skip and the bias once for all), all its loads are issued before the first
// is used, and the S / 4 lanes of a channel add up C h.  U = 4 where that leaves two blocks an SM (fewer reads of A, more
// bytes in flight), else 1 (more threads).
#include "la_ssm.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float4 four(const __nv_bfloat16 *a) {
    const uint2 v = *reinterpret_cast<const uint2 *>(a);
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xffff0000u));
}
__device__ __forceinline__ float4 four(const float *a) { return *reinterpret_cast<const float4 *>(a); }

template <typename T, int S, int U>
__global__ void __launch_bounds__(kThreads) k_ssm_step(SsmStepParams p) {
    constexpr int LPC = S / 4, CH = kThreads / LPC;
    pdl_wait();
    const int tiles = (p.E + CH - 1) / CH;
    const int b0 = blockIdx.x / tiles * U, e = blockIdx.x % tiles * CH + threadIdx.x / LPC, r = threadIdx.x % LPC;
    const bool there = e < p.E;
    const int ch = there ? e : 0, grp = ch / p.Eg;
    int slot[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int b = min(b0 + i, p.nB - 1);
        slot[i] = p.slots ? p.slots[b] : b;
        if (slot[i] >= p.pool) slot[i] = -1;
    }
    const float4 A = *reinterpret_cast<const float4 *>(p.A + (size_t)ch * S + 4 * r);
    const float bias = p.dt_bias ? p.dt_bias[ch] : 0.f, skip = p.skip ? p.skip[ch] : 0.f;
    float4 h[U], B[U], C[U];
    T x[U], v[U], z[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const long long b = min(b0 + i, p.nB - 1);
        x[i] = static_cast<const T *>(p.x)[b * p.sx.b + ch];
        v[i] = static_cast<const T *>(p.dt)[b * p.sdt.b + ch];
        z[i] = p.z ? static_cast<const T *>(p.z)[b * p.sz.b + ch] : x[i];
        B[i] = four(static_cast<const T *>(p.B) + b * p.sB.b + grp * p.sB.h + 4 * r);
        C[i] = four(static_cast<const T *>(p.C) + b * p.sC.b + grp * p.sC.h + 4 * r);
        h[i] = slot[i] < 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                           : *reinterpret_cast<const float4 *>(p.state + ((size_t)slot[i] * p.E + ch) * S + 4 * r);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const float dv = to_f32(v[i]) + bias, xi = to_f32(x[i]), zi = to_f32(z[i]);
        float ev;
        const float d = p.softplus ? softplus(dv, ev) : dv, d2 = d * kLog2e, u = d * xi;
        const float4 n = make_float4(fmaf(ex2(d2 * A.x), h[i].x, u * B[i].x), fmaf(ex2(d2 * A.y), h[i].y, u * B[i].y),
                                     fmaf(ex2(d2 * A.z), h[i].z, u * B[i].z), fmaf(ex2(d2 * A.w), h[i].w, u * B[i].w));
        float y = fmaf(n.x, C[i].x, fmaf(n.y, C[i].y, fmaf(n.z, C[i].z, n.w * C[i].w)));
#pragma unroll
        for (int m = 1; m < LPC; m <<= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
        if (!there || b0 + i >= p.nB) continue;
        if (slot[i] >= 0) *reinterpret_cast<float4 *>(p.state_out + ((size_t)slot[i] * p.E + ch) * S + 4 * r) = n;
        y = fmaf(skip, xi, y);
        if (p.z) y *= zi * sigmoid(zi);
        if (r == 0) static_cast<T *>(p.out)[(size_t)(b0 + i) * p.E + ch] = from_f32<T>(slot[i] < 0 ? 0.f : y);
    }
}

template <typename T, int S>
cudaError_t step_s(const SsmStepParams &p, cudaStream_t s) {
    TraceScope tr("ssm_step", s);
    const int CH = kThreads / (S / 4);
    const long long tiles = (p.E + CH - 1) / CH, wide = tiles * ((p.nB + 3) / 4);
    if (wide >= 2 * kPlanSms) return launch_pdl(k_ssm_step<T, S, 4>, dim3((unsigned)wide), dim3(kThreads), 0, s, p);
    return launch_pdl(k_ssm_step<T, S, 1>, dim3((unsigned)(tiles * p.nB)), dim3(kThreads), 0, s, p);
}

template <typename T>
cudaError_t step_t(const SsmStepParams &p, cudaStream_t s) {
    return p.S == 8 ? step_s<T, 8>(p, s) : p.S == 16 ? step_s<T, 16>(p, s) : p.S == 32 ? step_s<T, 32>(p, s) : step_s<T, 64>(p, s);
}

}  // namespace

cudaError_t ssm_step(const SsmStepParams &p, la_dtype dt, cudaStream_t s) {
    return dt == LA_BF16 ? step_t<__nv_bfloat16>(p, s) : step_t<float>(p, s);
}

}  // namespace la
