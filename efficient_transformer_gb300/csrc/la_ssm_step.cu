// la_ssm_step.cu -- selective state space scan, one token of each sequence on a pool of states.
//
//   h <- exp(d A) h + d x B,   out = (C . h + skip x) z sigmoid(z)
//
// Bound by memory: a state is read and written once for 4 operations and an ex2.  A thread holds 8 states of one channel for
// each of U sequences (A, skip and the bias once for all; with 4 states a lane the preparation, which a channel's lanes all
// do, was most of the instructions), all its loads are issued before the first is used, and the S / 8 lanes of the channel
// add up C h.  U = 2 where that leaves four blocks an SM (fewer reads of A, more bytes in flight), else 1 (more threads).
// 192 sequences of 4096 x 16, bfloat16: 22.3 us a call, 4.8 TB/s.  All decays have the slow states' correction (la_ssm.cuh): to
// choose it by the step, as the scan does, took 6 % more.
#include "la_ssm.cuh"

namespace la {
namespace {

constexpr int kThreads = 128;

// Eight elements in a row as they lie, widened where they are used.
template <typename T>
struct Raw8 {
    uint4 v[sizeof(T) / 2];
    __device__ __forceinline__ void get(const T *a) {
#pragma unroll
        for (int i = 0; i < (int)sizeof(T) / 2; ++i) v[i] = reinterpret_cast<const uint4 *>(a)[i];
    }
    __device__ __forceinline__ F2 pair(int i) const {   // elements 2 i and 2 i + 1
        if (sizeof(T) == 2) {
            const unsigned w = i == 0 ? v[0].x : i == 1 ? v[0].y : i == 2 ? v[0].z : v[0].w;
            return F2{__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)};
        }
        const uint4 &q = v[i / 2 % (sizeof(T) / 2)];
        return i % 2 ? F2{__uint_as_float(q.z), __uint_as_float(q.w)} : F2{__uint_as_float(q.x), __uint_as_float(q.y)};
    }
};

template <typename T, int S, int U>
__global__ void __launch_bounds__(kThreads) k_ssm_step(SsmStepParams p) {
    constexpr int LPC = S / 8, CH = kThreads / LPC;
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
    const size_t at = (size_t)ch * S + 8 * r, one = (size_t)p.E * S;
    Raw8<float> A, h[U];
    A.get(p.A + at);
    const float bias = p.dt_bias ? p.dt_bias[ch] : 0.f, skip = p.skip ? p.skip[ch] : 0.f;
    Raw8<T> B[U], C[U];
    T x[U], v[U], z[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const long long b = min(b0 + i, p.nB - 1);
        x[i] = (static_cast<const T *>(p.x) + b * p.sx.b)[ch];
        v[i] = (static_cast<const T *>(p.dt) + b * p.sdt.b)[ch];
        z[i] = p.z ? (static_cast<const T *>(p.z) + b * p.sz.b)[ch] : x[i];
        B[i].get(static_cast<const T *>(p.B) + b * p.sB.b + grp * p.sB.h + 8 * r);
        C[i].get(static_cast<const T *>(p.C) + b * p.sC.b + grp * p.sC.h + 8 * r);
        h[i] = Raw8<float>{};
        if (slot[i] >= 0) h[i].get(p.state + slot[i] * one + at);
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const float dv = to_f32(v[i]) + bias, xi = to_f32(x[i]), zi = to_f32(z[i]);
        float ev;
        const float d = p.softplus ? softplus(dv, ev) : dv;
        const F2 d2 = f2(d * kLog2e), u = f2(d * xi);
        F2 n[4], acc;
#pragma unroll
        for (int m = 0; m < 4; ++m) {
            n[m] = fma2(decay2(d2, A.pair(m), f2(kTiltSlow)), h[i].pair(m), mul2(u, B[i].pair(m)));
            acc = m == 0 ? mul2(n[m], C[i].pair(m)) : fma2(n[m], C[i].pair(m), acc);
        }
        float y = acc.x + acc.y;
#pragma unroll
        for (int m = 1; m < LPC; m <<= 1) y += __shfl_xor_sync(0xffffffffu, y, m);
        if (!there || b0 + i >= p.nB) continue;
        if (slot[i] >= 0) {
            float4 *to = reinterpret_cast<float4 *>(p.state_out + slot[i] * one + at);
            to[0] = make_float4(n[0].x, n[0].y, n[1].x, n[1].y);
            to[1] = make_float4(n[2].x, n[2].y, n[3].x, n[3].y);
        }
        y = fmaf(skip, xi, y);
        if (p.z) y *= zi * sigmoid(zi);
        if (r == 0) static_cast<T *>(p.out)[(size_t)(b0 + i) * p.E + ch] = from_f32<T>(slot[i] < 0 ? 0.f : y);
    }
}

template <typename T, int S>
cudaError_t step_s(const SsmStepParams &p, cudaStream_t s) {
    TraceScope tr("ssm_step", s);
    const int CH = kThreads / (S / 8);
    const long long tiles = (p.E + CH - 1) / CH, wide = tiles * ((p.nB + 1) / 2);
    if (wide >= 4 * kPlanSms) return launch_pdl(k_ssm_step<T, S, 2>, dim3((unsigned)wide), dim3(kThreads), 0, s, p);
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
