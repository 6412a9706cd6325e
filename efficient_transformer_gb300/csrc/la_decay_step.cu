// la_decay_step.cu -- decayed linear attention, recurrent form: one token of each sequence.
//
//   S <- gamma S + k v^T,   out_h = scale q_h^T S   for the n_rep query heads h of the group
//
// Bound by memory: a state of D x Dv floats is read and written once for 2 (1 + n_rep) D Dv flop.  A
// block owns COLS columns of one head's state; a thread holds the rows of its group, 4 columns wide, in
// registers, all loaded before the first is used, and sums q S over its rows; the row groups meet
// in the warp and then in shared memory.  COLS = Dv where that gives every SM a few blocks (whole rows,
// q and k fetched once a head), 32 where there are few heads and the blocks' number counts (192 sequences of 32/8
// heads, 128 x 128: 36 us, 5.6 TB/s; with 32 columns 44 us).
#include "la_decay.cuh"

namespace la {
namespace {

constexpr int kThreads = 256;
constexpr int kHeads = 8;   // query heads summed per trip

template <typename T, int D, int COLS>
__global__ void __launch_bounds__(kThreads) k_decay_step(DecayStepParams p) {
    constexpr int L = COLS / 4, RG = kThreads / L, R = D / RG;   // lanes a row, row groups, rows a thread
    constexpr int W = L < 32 ? kThreads / 32 : RG;               // partial sums of a column after the warps
    __shared__ float part[W][kHeads][COLS];
    __shared__ float ks[D], qs[kHeads][D];
    pdl_wait();
    const int slabs = p.Dv / COLS;
    const int slab = blockIdx.x % slabs, bg = blockIdx.x / slabs, b = bg / p.Hkv, h = bg % p.Hkv;
    const int lane = threadIdx.x % L, rg = threadIdx.x / L, c = slab * COLS + lane * 4;
    T *out = static_cast<T *>(p.out) + ((size_t)b * p.Hkv + h) * p.n_rep * p.Dv + slab * COLS;
    const int slot = p.slots ? p.slots[b] : b;
    if (slot < 0 || slot >= p.pool) {
        for (int i = threadIdx.x; i < p.n_rep * COLS; i += kThreads) out[(i / COLS) * p.Dv + i % COLS] = from_f32<T>(0.f);
        return;
    }
    // rows rg, rg + RG, ...
    const size_t base = ((size_t)slot * p.Hkv + h) * D * p.Dv + c;
    float4 S[R];
#pragma unroll
    for (int m = 0; m < R; ++m) S[m] = *reinterpret_cast<const float4 *>(p.state + base + (size_t)(rg + m * RG) * p.Dv);
    const T *k = static_cast<const T *>(p.k) + b * p.sk.b + h * p.sk.h;
    const T *q = static_cast<const T *>(p.q) + b * p.sq.b + (long long)h * p.n_rep * p.sq.h;
    const T *v = static_cast<const T *>(p.v) + b * p.sv.b + h * p.sv.h + c;
    for (int d = threadIdx.x; d < D; d += kThreads) ks[d] = to_f32(k[d]);
    const float g = exp2f(decay_log2(p.log_decay[h]));
    const float4 vv = make_float4(to_f32(v[0]), to_f32(v[1]), to_f32(v[2]), to_f32(v[3]));
    for (int r0 = 0; r0 < p.n_rep; r0 += kHeads) {
        const int nr = min(kHeads, p.n_rep - r0);
        for (int i = threadIdx.x; i < nr * D; i += kThreads) qs[i / D][i % D] = to_f32(q[(r0 + i / D) * p.sq.h + i % D]);
        __syncthreads();
        if (r0 == 0) {
#pragma unroll
            for (int m = 0; m < R; ++m) {
                const float kd = ks[rg + m * RG];
                S[m] = make_float4(fmaf(g, S[m].x, kd * vv.x), fmaf(g, S[m].y, kd * vv.y), fmaf(g, S[m].z, kd * vv.z),
                                   fmaf(g, S[m].w, kd * vv.w));
                *reinterpret_cast<float4 *>(p.state_out + base + (size_t)(rg + m * RG) * p.Dv) = S[m];
            }
        }
        for (int r = 0; r < nr; ++r) {
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int m = 0; m < R; ++m) {
                const float qd = qs[r][rg + m * RG];
                o.x = fmaf(qd, S[m].x, o.x);
                o.y = fmaf(qd, S[m].y, o.y);
                o.z = fmaf(qd, S[m].z, o.z);
                o.w = fmaf(qd, S[m].w, o.w);
            }
#pragma unroll
            for (int d = L; d < 32; d *= 2) {
                o.x += __shfl_xor_sync(0xffffffffu, o.x, d);
                o.y += __shfl_xor_sync(0xffffffffu, o.y, d);
                o.z += __shfl_xor_sync(0xffffffffu, o.z, d);
                o.w += __shfl_xor_sync(0xffffffffu, o.w, d);
            }
            if (threadIdx.x % 32 < L) *reinterpret_cast<float4 *>(&part[threadIdx.x / 32][r][lane * 4]) = o;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < nr * COLS; i += kThreads) {
            const int r = i / COLS, e = i % COLS;
            float o = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) o += part[w][r][e];
            out[(size_t)(r0 + r) * p.Dv + e] = from_f32<T>(p.scale * o);
        }
    }
}

template <typename T, int COLS>
cudaError_t step_c(const DecayStepParams &p, cudaStream_t s) {
    TraceScope tr("decay_step", s);
    auto kern = p.D == 32 ? k_decay_step<T, 32, COLS> : p.D == 64 ? k_decay_step<T, 64, COLS> : k_decay_step<T, 128, COLS>;
    return launch_pdl(kern, dim3((unsigned)p.B * p.Hkv * (p.Dv / COLS)), dim3(kThreads), 0, s, p);
}

template <typename T>
cudaError_t step_t(const DecayStepParams &p, cudaStream_t s) {
    if (p.Dv == 32 || p.B * p.Hkv < 4 * kPlanSms) return step_c<T, 32>(p, s);
    return p.Dv == 64 ? step_c<T, 64>(p, s) : step_c<T, 128>(p, s);
}

}  // namespace

cudaError_t decay_step(const DecayStepParams &p, la_dtype dt, cudaStream_t s) {
    return dt == LA_BF16 ? step_t<__nv_bfloat16>(p, s) : step_t<float>(p, s);
}

}  // namespace la
