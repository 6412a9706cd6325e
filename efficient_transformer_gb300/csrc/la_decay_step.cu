// la_decay_step.cu -- decayed linear attention, recurrent form: one token of each sequence.
//
//   S <- gamma S + k v^T,   out_h = scale q_h^T S   for the n_rep query heads h of the group
//
// Bound by memory: a state of D x Dv floats is read and written once for 2 (1 + n_rep) D Dv flop.  A
// block owns kCols columns of one head's state; a thread holds D / kRowGroups rows of 4 columns in
// registers, all loaded before the first is used, and sums q S over its rows; the row groups meet
// in the warp and then in shared memory.
#include "la_decay.cuh"

namespace la {
namespace {

constexpr int kThreads = 256, kCols = 32, kLanes = kCols / 4, kRowGroups = kThreads / kLanes;
constexpr int kHeads = 8;   // query heads summed per trip (registers)

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) k_decay_step(DecayStepParams p) {
    constexpr int R = D / kRowGroups;
    __shared__ float part[kThreads / 32][kHeads][kCols];
    pdl_wait();
    const int slabs = p.Dv / kCols;
    const int slab = blockIdx.x % slabs, bg = blockIdx.x / slabs, b = bg / p.Hkv, h = bg % p.Hkv;
    const int lane = threadIdx.x % kLanes, rg = threadIdx.x / kLanes, c = slab * kCols + lane * 4;
    T *out = static_cast<T *>(p.out) + ((size_t)b * p.Hkv + h) * p.n_rep * p.Dv + slab * kCols;
    const int slot = p.slots ? p.slots[b] : b;
    if (slot < 0 || slot >= p.pool) {
        for (int i = threadIdx.x; i < p.n_rep * kCols; i += kThreads) out[(i / kCols) * p.Dv + i % kCols] = from_f32<T>(0.f);
        return;
    }
    const size_t base = ((size_t)slot * p.Hkv + h) * D * p.Dv + c;
    float4 S[R];
#pragma unroll
    for (int m = 0; m < R; ++m) S[m] = *reinterpret_cast<const float4 *>(p.state + base + (size_t)(rg + m * kRowGroups) * p.Dv);
    const T *k = static_cast<const T *>(p.k) + b * p.sk.b + h * p.sk.h;
    const T *v = static_cast<const T *>(p.v) + b * p.sv.b + h * p.sv.h + c;
    const float g = exp2f(decay_log2(p.log_decay[h]));
    const float4 vv = make_float4(to_f32(v[0]), to_f32(v[1]), to_f32(v[2]), to_f32(v[3]));
#pragma unroll
    for (int m = 0; m < R; ++m) {
        const float kd = to_f32(k[rg + m * kRowGroups]);
        S[m] = make_float4(fmaf(g, S[m].x, kd * vv.x), fmaf(g, S[m].y, kd * vv.y), fmaf(g, S[m].z, kd * vv.z),
                           fmaf(g, S[m].w, kd * vv.w));
        *reinterpret_cast<float4 *>(p.state_out + base + (size_t)(rg + m * kRowGroups) * p.Dv) = S[m];
    }
    for (int r0 = 0; r0 < p.n_rep; r0 += kHeads) {
        const int nr = min(kHeads, p.n_rep - r0);
        for (int r = 0; r < nr; ++r) {
            const T *q = static_cast<const T *>(p.q) + b * p.sq.b + ((long long)h * p.n_rep + r0 + r) * p.sq.h;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int m = 0; m < R; ++m) {
                const float qd = to_f32(q[rg + m * kRowGroups]);
                o.x = fmaf(qd, S[m].x, o.x);
                o.y = fmaf(qd, S[m].y, o.y);
                o.z = fmaf(qd, S[m].z, o.z);
                o.w = fmaf(qd, S[m].w, o.w);
            }
#pragma unroll
            for (int d = kLanes; d < 32; d *= 2) {
                o.x += __shfl_xor_sync(0xffffffffu, o.x, d);
                o.y += __shfl_xor_sync(0xffffffffu, o.y, d);
                o.z += __shfl_xor_sync(0xffffffffu, o.z, d);
                o.w += __shfl_xor_sync(0xffffffffu, o.w, d);
            }
            if (threadIdx.x % 32 < kLanes) *reinterpret_cast<float4 *>(&part[threadIdx.x / 32][r][lane * 4]) = o;
        }
        __syncthreads();
        if (threadIdx.x < nr * kCols) {
            const int r = threadIdx.x / kCols, e = threadIdx.x % kCols;
            float o = 0.f;
#pragma unroll
            for (int w = 0; w < kThreads / 32; ++w) o += part[w][r][e];
            out[(size_t)(r0 + r) * p.Dv + e] = from_f32<T>(p.scale * o);
        }
        if (r0 + kHeads < p.n_rep) __syncthreads();
    }
}

template <typename T>
cudaError_t step_t(const DecayStepParams &p, cudaStream_t s) {
    TraceScope tr("decay_step", s);
    auto kern = p.D == 32 ? k_decay_step<T, 32> : p.D == 64 ? k_decay_step<T, 64> : k_decay_step<T, 128>;
    return launch_pdl(kern, dim3((unsigned)p.B * p.Hkv * (p.Dv / kCols)), dim3(kThreads), 0, s, p);
}

}  // namespace

cudaError_t decay_step(const DecayStepParams &p, la_dtype dt, cudaStream_t s) {
    return dt == LA_BF16 ? step_t<__nv_bfloat16>(p, s) : step_t<float>(p, s);
}

}  // namespace la
