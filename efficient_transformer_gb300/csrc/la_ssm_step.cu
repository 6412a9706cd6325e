// la_ssm_step.cu -- selective state space scan, one token of each sequence on a pool of states.
//
//   h <- exp(d A) h + d x B,   out = (C . h + skip x) z sigmoid(z)
//
// Bound by memory: a state is read and written once for 4 operations and an ex2.  A thread holds 4 states of a channel
// (one 16-byte load), all its other loads are issued beside it, and the S / 4 lanes of the channel add up C h.
#include "la_ssm.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;

template <typename T, int S>
__global__ void __launch_bounds__(kThreads) k_ssm_step(SsmStepParams p) {
    constexpr int LPC = S / 4, CH = kThreads / LPC;
    pdl_wait();
    const int tiles = (p.E + CH - 1) / CH;
    const int b = blockIdx.x / tiles, e = blockIdx.x % tiles * CH + threadIdx.x / LPC, r = threadIdx.x % LPC;
    const bool there = e < p.E;
    const int ch = there ? e : 0, grp = ch / p.Eg;
    const int slot = p.slots ? p.slots[b] : b;
    T *out = static_cast<T *>(p.out) + (size_t)b * p.E + ch;
    if (slot < 0 || slot >= p.pool) {
        if (there && r == 0) *out = from_f32<T>(0.f);
        return;
    }
    const size_t at = ((size_t)slot * p.E + ch) * S + 4 * r;
    const float4 h = *reinterpret_cast<const float4 *>(p.state + at);
    const float4 A = *reinterpret_cast<const float4 *>(p.A + (size_t)ch * S + 4 * r);
    const float x = to_f32(static_cast<const T *>(p.x)[b * p.sx.b + ch]);
    const float v = to_f32(static_cast<const T *>(p.dt)[b * p.sdt.b + ch]) + (p.dt_bias ? p.dt_bias[ch] : 0.f);
    const float z = p.z ? to_f32(static_cast<const T *>(p.z)[b * p.sz.b + ch]) : 0.f;
    const float skip = p.skip ? p.skip[ch] : 0.f;
    const T *Bp = static_cast<const T *>(p.B) + b * p.sB.b + grp * p.sB.h + 4 * r;
    const T *Cp = static_cast<const T *>(p.C) + b * p.sC.b + grp * p.sC.h + 4 * r;
    const float4 B = make_float4(to_f32(Bp[0]), to_f32(Bp[1]), to_f32(Bp[2]), to_f32(Bp[3]));
    const float4 C = make_float4(to_f32(Cp[0]), to_f32(Cp[1]), to_f32(Cp[2]), to_f32(Cp[3]));
    float ev;
    const float d = p.softplus ? softplus(v, ev) : v, d2 = d * kLog2e, u = d * x;
    const float4 n = make_float4(fmaf(ex2(d2 * A.x), h.x, u * B.x), fmaf(ex2(d2 * A.y), h.y, u * B.y),
                                 fmaf(ex2(d2 * A.z), h.z, u * B.z), fmaf(ex2(d2 * A.w), h.w, u * B.w));
    if (there) *reinterpret_cast<float4 *>(p.state_out + at) = n;
    float y = fmaf(n.x, C.x, fmaf(n.y, C.y, fmaf(n.z, C.z, n.w * C.w)));
#pragma unroll
    for (int m = 1; m < LPC; m <<= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
    y = fmaf(skip, x, y);
    if (p.z) y *= z * sigmoid(z);
    if (there && r == 0) *out = from_f32<T>(y);
}

template <typename T>
cudaError_t step_t(const SsmStepParams &p, cudaStream_t s) {
    TraceScope tr("ssm_step", s);
    const int CH = kThreads / (p.S / 4);
    auto kern = p.S == 8 ? k_ssm_step<T, 8> : p.S == 16 ? k_ssm_step<T, 16> : p.S == 32 ? k_ssm_step<T, 32> : k_ssm_step<T, 64>;
    return launch_pdl(kern, dim3((unsigned)((long long)((p.E + CH - 1) / CH) * p.nB)), dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t ssm_step(const SsmStepParams &p, la_dtype dt, cudaStream_t s) {
    return dt == LA_BF16 ? step_t<__nv_bfloat16>(p, s) : step_t<float>(p, s);
}

}  // namespace la
