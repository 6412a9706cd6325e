// la_conv.cu -- short causal convolution of every channel with W taps, with silu or without: forward, gradient, single
// token, and their C ABI.
//
//   v_t = bias + sum_j w_j x_(t - W + 1 + j),   out_t = v_t sigmoid(v_t)
//   g'_t = g_t (v sigmoid(v))',   dx_t = sum_j w_j g'_(t + W - 1 - j),   dw_j = sum_t g'_t x_(t - W + 1 + j),   db = sum g'
//
// Bound by memory: each row is read once but for the W - 1 rows at a run's edge.  A thread owns a few channels (one vector load
// a token) and walks a run of tokens with the last W rows in registers; the loads of several tokens are issued together.
#include <initializer_list>

#include "la_internal.cuh"

namespace la {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

struct ConvParams {
    const void *x, *g, *weight, *bias, *init, *dfinal;
    Strides sx, sg;
    const int *lengths, *slots;
    void *out, *fin, *dinit, *dweight, *dbias;
    float *part;                  // gradient: [parts][W + 1][E]
    int B, N, E, silu, wide;      // wide: weight and bias are float32
    int run, runs, parts, pool;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float sigmoid(float v) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(1.f + ex2(-v * kLog2e)));
    return y;
}

// V channels of a row
template <typename T, int V>
struct __align__(sizeof(T) * V) Row {
    T v[V];
};
template <typename T, int V>
__device__ __forceinline__ Row<T, V> no_row() {
    Row<T, V> r;
#pragma unroll
    for (int c = 0; c < V; ++c) r.v[c] = from_f32<T>(0.f);
    return r;
}
template <typename T, int V>
__device__ __forceinline__ Row<T, V> get_row(const void *base, long long at) {
    return *reinterpret_cast<const Row<T, V> *>(static_cast<const T *>(base) + at);
}
template <typename T, int V>
__device__ __forceinline__ void put_row(void *base, long long at, const Row<T, V> &r) {
    *reinterpret_cast<Row<T, V> *>(static_cast<T *>(base) + at) = r;
}

// n (a multiple of 4) float32 or T parameters in a row
template <typename T, int n>
__device__ __forceinline__ void get_parameters(float (&to)[n], const void *p, long long i, int wide) {
#pragma unroll
    for (int q = 0; q < n; q += 4) {
        if (wide) {
            const Row<float, 4> r = get_row<float, 4>(p, i + q);
#pragma unroll
            for (int c = 0; c < 4; ++c) to[q + c] = r.v[c];
        } else {
            const Row<T, 4> r = get_row<T, 4>(p, i + q);
#pragma unroll
            for (int c = 0; c < 4; ++c) to[q + c] = to_f32(r.v[c]);
        }
    }
}

template <typename T, int W, int V>
struct Taps {
    float w[V * W], bias[V];      // w: channel by channel, as it lies
    __device__ __forceinline__ Taps(const ConvParams &p, int e) {
        get_parameters<T>(w, p.weight, (long long)e * W, p.wide);
#pragma unroll
        for (int c = 0; c < V; ++c) bias[c] = 0.f;
        if (p.bias) get_parameters<T>(bias, p.bias, e, p.wide);
    }
    __device__ __forceinline__ float at(int j, int c) const { return w[c * W + j]; }
};

constexpr int kBatch = 8;         // tokens whose loads are issued together

// Forward.  Thread: V channels, `run` tokens (a multiple of kBatch) of one sequence.
template <typename T, int W>
__global__ void __launch_bounds__(256) k_conv(ConvParams p) {
    constexpr int V = 16 / (int)sizeof(T);
    pdl_wait();
    const int vecs = p.E / V;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= (long long)p.B * p.runs * vecs) return;
    const int e = (int)(i % vecs) * V, run = (int)(i / vecs % p.runs), b = (int)(i / vecs / p.runs);
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.N) : p.N;
    const int t0 = run * p.run, t1 = min(t0 + p.run, p.N), te = min(t1, len);
    const Taps<T, W, V> k(p, e);
    const long long x0 = b * p.sx.b + e, o0 = (long long)b * p.N * p.E + e, s0 = (long long)b * (W - 1) * p.E + e;
    auto before = [&](int t) {    // row t of the sequence with the W - 1 inputs before its first
        if (t >= 0) return get_row<T, V>(p.x, x0 + t * p.sx.n);
        return p.init ? get_row<T, V>(p.init, s0 + (long long)(t + W - 1) * p.E) : no_row<T, V>();
    };
    float win[W][V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const Row<T, V> r = t0 < te ? before(t0 - (W - 1) + j) : no_row<T, V>();
#pragma unroll
        for (int c = 0; c < V; ++c) win[j + 1][c] = to_f32(r.v[c]);
    }
    // The first run's thread alone reads the initial state; having read it, it writes the final one, which may take its place.
    if (run == 0 && p.fin) {
        Row<T, V> last[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) last[j] = before(len - (W - 1) + j);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) put_row<T, V>(p.fin, s0 + (long long)j * p.E, last[j]);
    }
    for (int t = t0; t < t1; t += kBatch) {
        Row<T, V> in[kBatch];
#pragma unroll
        for (int q = 0; q < kBatch; ++q) in[q] = t + q < te ? get_row<T, V>(p.x, x0 + (t + q) * p.sx.n) : no_row<T, V>();
#pragma unroll
        for (int q = 0; q < kBatch; ++q) {
            Row<T, V> o;
#pragma unroll
            for (int c = 0; c < V; ++c) {
#pragma unroll
                for (int j = 0; j < W - 1; ++j) win[j][c] = win[j + 1][c];
                win[W - 1][c] = to_f32(in[q].v[c]);
                float v = k.bias[c];
#pragma unroll
                for (int j = 0; j < W; ++j) v = fmaf(k.at(j, c), win[j][c], v);
                if (p.silu) v *= sigmoid(v);
                o.v[c] = from_f32<T>(t + q < te ? v : 0.f);
            }
            if (t + q < t1) put_row<T, V>(p.out, o0 + (long long)(t + q) * p.E, o);
        }
    }
}

// Gradient.  Block: 32 x V channels, 8 runs of one sequence; dw and db of a thread's run are added up over the block.
// Half the forward's channels a thread: three windows of W rows are held beside the taps.
template <typename T, int W>
__global__ void __launch_bounds__(256) k_conv_grad(ConvParams p) {
    constexpr int V = 4, Q = 4;
    __shared__ float sums[8][W + 1][32 * V];
    pdl_wait();
    const int tiles = (p.E + 32 * V - 1) / (32 * V), groups = (p.runs + 7) / 8;
    const int tile = blockIdx.x % tiles, grp = blockIdx.x / tiles % groups, b = blockIdx.x / tiles / groups;
    const int lane = threadIdx.x % 32, y = threadIdx.x / 32, e = (tile * 32 + lane) * V, run = grp * 8 + y;
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.N) : p.N;
    const int t0 = run * p.run, t1 = min(t0 + p.run, p.N);
    float dw[W][V], db[V];
#pragma unroll
    for (int c = 0; c < V; ++c) {
        db[c] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][c] = 0.f;
    }
    if (e < p.E && t0 < p.N) {
        const Taps<T, W, V> k(p, e);
        const long long x0 = b * p.sx.b + e, g0 = b * p.sg.b + e, o0 = (long long)b * p.N * p.E + e,
                        s0 = (long long)b * (W - 1) * p.E + e;
        float win[W][V], gw[W][V];   // rows x_(t - W + 1 ..  t) and g'_(t - W + 1 .. t)
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int c = 0; c < V; ++c) gw[j][c] = 0.f;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const int t = t0 - (W - 1) + j;
            const Row<T, V> r = t >= 0 ? (t < len ? get_row<T, V>(p.x, x0 + t * p.sx.n) : no_row<T, V>())
                                       : p.init ? get_row<T, V>(p.init, s0 + (long long)(t + W - 1) * p.E) : no_row<T, V>();
#pragma unroll
            for (int c = 0; c < V; ++c) win[j + 1][c] = to_f32(r.v[c]);
        }
        // token t gives g'_t and with it the gradient of row t - W + 1; the first run starts with the rows before the first
        // token, the others end W - 1 tokens past their run
        for (int t = t0; t < t1 + W - 1; t += Q) {
            Row<T, V> in[Q], gin[Q];
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const bool in_len = t + q < len;
                in[q] = in_len ? get_row<T, V>(p.x, x0 + (t + q) * p.sx.n) : no_row<T, V>();
                gin[q] = in_len ? get_row<T, V>(p.g, g0 + (t + q) * p.sg.n) : no_row<T, V>();
            }
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                const int at = t + q - (W - 1);   // the row whose gradient is whole now
                const bool mine = t + q < t1;
                float dx[V];
#pragma unroll
                for (int c = 0; c < V; ++c) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) {
                        win[j][c] = win[j + 1][c];
                        gw[j][c] = gw[j + 1][c];
                    }
                    win[W - 1][c] = to_f32(in[q].v[c]);
                    float g = to_f32(gin[q].v[c]);
                    if (p.silu) {
                        float v = k.bias[c];
#pragma unroll
                        for (int j = 0; j < W; ++j) v = fmaf(k.at(j, c), win[j][c], v);
                        const float s = sigmoid(v);
                        g *= s * fmaf(v, 1.f - s, 1.f);
                        g = t + q < len ? g : 0.f;
                    }
                    gw[W - 1][c] = g;
                    if (mine) {
                        db[c] += g;
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][c] = fmaf(g, win[j][c], dw[j][c]);
                    }
                    float s = 0.f;
#pragma unroll
                    for (int j = 0; j < W; ++j) s = fmaf(k.at(j, c), gw[W - 1 - j][c], s);
                    dx[c] = s;
                }
                // (a thread's first W - 1 rows are whole in the run before, but for those in front of the first token)
                const bool front = at < 0;
                if (at >= t1 || (front ? run != 0 || !p.dinit : at < t0)) continue;
                const int f = at + (W - 1) - len;   // the row's place in the final state
                Row<T, V> o, add = no_row<T, V>();
                if (p.dfinal && f >= 0 && f < W - 1) add = get_row<T, V>(p.dfinal, s0 + (long long)f * p.E);
#pragma unroll
                for (int c = 0; c < V; ++c) o.v[c] = from_f32<T>(at < len ? dx[c] + to_f32(add.v[c]) : 0.f);
                if (front) put_row<T, V>(p.dinit, s0 + (long long)(at + W - 1) * p.E, o);
                else put_row<T, V>(p.out, o0 + (long long)at * p.E, o);
            }
        }
    }
#pragma unroll
    for (int c = 0; c < V; ++c) {
#pragma unroll
        for (int j = 0; j < W; ++j) sums[y][j][lane * V + c] = dw[j][c];
        sums[y][W][lane * V + c] = db[c];
    }
    __syncthreads();
    float *part = p.part + (size_t)(b * groups + grp) * (W + 1) * p.E;
    for (int i = threadIdx.x; i < (W + 1) * 32 * V; i += 256) {
        const int j = i / (32 * V), c = i % (32 * V);
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) s += sums[q][j][c];
        if (tile * 32 * V + c < p.E) part[(size_t)j * p.E + tile * 32 * V + c] = s;
    }
}

// dw [E, W] and db [E] from the blocks' parts, in a fixed order: 8 threads a value, each an eighth of the parts.
template <typename T>
__global__ void __launch_bounds__(256) k_conv_reduce(ConvParams p, int W) {
    __shared__ float sums[8][32];
    pdl_wait();
    const int lane = threadIdx.x % 32, y = threadIdx.x / 32;
    const long long i = (long long)blockIdx.x * 32 + lane, n = (long long)(W + 1) * p.E;
    float s = 0.f;
    if (i < n)
        for (int q = y; q < p.parts; q += 8) s += p.part[(size_t)q * n + i];
    sums[y][lane] = s;
    __syncthreads();
    if (y != 0 || i >= n) return;
#pragma unroll
    for (int q = 1; q < 8; ++q) s += sums[q][lane];
    const int j = (int)(i / p.E), e = (int)(i % p.E);
    void *to = j < W ? p.dweight : p.dbias;
    const long long at = j < W ? (long long)e * W + j : e;
    if (!to) return;
    if (p.wide) static_cast<float *>(to)[at] = s;
    else static_cast<T *>(to)[at] = from_f32<T>(s);
}

// One token of each sequence; a state's W - 1 rows move up by one.
template <typename T, int W>
__global__ void __launch_bounds__(128) k_conv_step(ConvParams p) {
    constexpr int V = 16 / (int)sizeof(T);
    pdl_wait();
    const int vecs = p.E / V;
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    if (i >= (long long)p.B * vecs) return;
    const int e = (int)(i % vecs) * V, b = (int)(i / vecs);
    const int slot = p.slots ? p.slots[b] : b;
    if (slot < 0 || slot >= p.pool) {
        put_row<T, V>(p.out, (long long)b * p.E + e, no_row<T, V>());
        return;
    }
    const long long s0 = (long long)slot * (W - 1) * p.E + e;
    Row<T, V> win[W], o;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j] = get_row<T, V>(p.init, s0 + (long long)j * p.E);
    win[W - 1] = get_row<T, V>(p.x, b * p.sx.b + e);
    const Taps<T, W, V> k(p, e);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) put_row<T, V>(p.fin, s0 + (long long)j * p.E, win[j + 1]);
#pragma unroll
    for (int c = 0; c < V; ++c) {
        float v = k.bias[c];
#pragma unroll
        for (int j = 0; j < W; ++j) v = fmaf(k.at(j, c), to_f32(win[j].v[c]), v);
        if (p.silu) v *= sigmoid(v);
        o.v[c] = from_f32<T>(v);
    }
    put_row<T, V>(p.out, (long long)b * p.E + e, o);
}

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Sizes and types; the weight's type is float32 or the inputs'.
la_status check(int B, int N, int E, int W, la_dtype dt, la_dtype wt) {
    if (B <= 0 || N <= 0 || E <= 0 || (dt != LA_F32 && dt != LA_BF16) || (wt != LA_F32 && wt != dt)) return LA_ERR_ARG;
    if (N > (1 << 30) || (long long)B * N > (1ll << 40)) return LA_ERR_ARG;
    if (W < 2 || W > 4 || E % 8) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

// Tokens of a forward thread: long runs read fewer rows twice, short ones give small inputs enough threads.
int forward_run(int B, int N, int E, la_dtype dt) {
    const long long rows = (long long)B * N * (E / (dt == LA_BF16 ? 8 : 4));
    int run = 64;
    while (run > kBatch && rows / run < (long long)kPlanSms * 2048) run /= 2;
    return run;
}
// ... and of a gradient thread: 8 runs are a block, which is one part of dw.
int grad_run(int B, int N, int E) {
    const long long rows = (long long)B * N * (E / 4);
    int run = 128;
    while (run > 8 && rows / run < (long long)kPlanSms * 1024) run /= 2;
    return run;
}
int grad_parts(int B, int N, int E) {
    const int run = grad_run(B, N, E), runs = (N + run - 1) / run;
    return B * ((runs + 7) / 8);
}

// Strides of a [B, N, E] input: 16-byte rows.
la_status strides_of(const la_strides *st, int B, int N, int E, la_dtype dt, Strides *out) {
    *out = Strides{(long long)N * E, 0, (long long)E};
    if (!st) return LA_OK;
    if (st->b < 0 || st->n < 0) return LA_ERR_ARG;
    if (B > 1) out->b = st->b;
    if (N > 1) out->n = st->n;
    const int unit = dt == LA_BF16 ? 8 : 4;
    return out->b % unit || out->n % unit ? LA_ERR_ALIGN : LA_OK;
}

la_status bad_pointers(std::initializer_list<const void *> vectors, const int *ints) {
    for (const void *p : vectors)
        if (p && !aligned(p, 16)) return LA_ERR_ALIGN;
    return ints && !aligned(ints, 4) ? LA_ERR_ALIGN : LA_OK;
}

template <typename T>
cudaError_t forward(const ConvParams &p, int W, cudaStream_t s) {
    TraceScope tr("conv", s);
    const long long threads = (long long)p.B * p.runs * (p.E / (16 / (int)sizeof(T)));
    auto kern = W == 2 ? k_conv<T, 2> : W == 3 ? k_conv<T, 3> : k_conv<T, 4>;
    return launch_pdl(kern, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, p);
}

template <typename T>
cudaError_t gradient(const ConvParams &p, int W, cudaStream_t s) {
    cudaError_t e;
    {
        TraceScope tr("conv_grad", s);
        const long long blocks = (long long)((p.E + 127) / 128) * ((p.runs + 7) / 8) * p.B;
        auto kern = W == 2 ? k_conv_grad<T, 2> : W == 3 ? k_conv_grad<T, 3> : k_conv_grad<T, 4>;
        e = launch_pdl(kern, dim3((unsigned)blocks), dim3(256), 0, s, p);
    }
    if (e != cudaSuccess) return e;
    TraceScope tr("conv_reduce", s);
    return launch_pdl(k_conv_reduce<T>, dim3((unsigned)(((long long)(W + 1) * p.E + 31) / 32)), dim3(256), 0, s, p, W);
}

template <typename T>
cudaError_t step(const ConvParams &p, int W, cudaStream_t s) {
    TraceScope tr("conv_step", s);
    const long long threads = (long long)p.B * (p.E / (16 / (int)sizeof(T)));
    auto kern = W == 2 ? k_conv_step<T, 2> : W == 3 ? k_conv_step<T, 3> : k_conv_step<T, 4>;
    return launch_pdl(kern, dim3((unsigned)((threads + 127) / 128)), dim3(128), 0, s, p);
}

}  // namespace
}  // namespace la

using namespace la;

extern "C" {

la_status la_conv_fwd(const void *x, const void *weight, const void *bias, void *out, const void *initial_state,
                      void *final_state, const int *lengths, int B, int N, int E, int W, la_dtype dtype,
                      la_dtype weight_dtype, int silu, const la_strides *x_strides, void *stream) {
    la_status st = check(B, N, E, W, dtype, weight_dtype);
    if (st != LA_OK) return st;
    if (!x || !weight || !out) return LA_ERR_ARG;
    if ((st = bad_pointers({x, weight, bias, out, initial_state, final_state}, lengths)) != LA_OK) return st;
    ConvParams p{};
    if ((st = strides_of(x_strides, B, N, E, dtype, &p.sx)) != LA_OK) return st;
    p.x = x; p.weight = weight; p.bias = bias; p.out = out; p.init = initial_state; p.fin = final_state;
    p.lengths = lengths; p.B = B; p.N = N; p.E = E; p.silu = silu; p.wide = weight_dtype == LA_F32;
    p.run = forward_run(B, N, E, dtype);
    p.runs = (N + p.run - 1) / p.run;
    if ((long long)B * p.runs * (E / 4) / 256 >= (1ll << 31) - 1) return LA_ERR_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = dtype == LA_BF16 ? forward<__nv_bfloat16>(p, W, s) : forward<float>(p, W, s);
    return e == cudaSuccess ? LA_OK : cuda_fail(e);
}

size_t la_conv_workspace_size(int B, int N, int E, int W, la_dtype dtype) {
    if (check(B, N, E, W, dtype, dtype) != LA_OK) return 0;
    return (size_t)grad_parts(B, N, E) * (W + 1) * E * 4;
}

la_status la_conv_bwd(const void *x, const void *weight, const void *bias, const void *grad_out, void *dx, void *dweight,
                      void *dbias, const void *initial_state, const void *grad_final_state, void *grad_initial_state,
                      const int *lengths, int B, int N, int E, int W, la_dtype dtype, la_dtype weight_dtype, int silu,
                      const la_strides *x_strides, const la_strides *g_strides, void *workspace, size_t ws_bytes,
                      void *stream) {
    la_status st = check(B, N, E, W, dtype, weight_dtype);
    if (st != LA_OK) return st;
    if (!x || !weight || !grad_out || !dx || !dweight || (dbias && !bias)) return LA_ERR_ARG;
    if (grad_initial_state && (grad_initial_state == initial_state || grad_initial_state == grad_final_state)) return LA_ERR_ARG;
    if ((st = bad_pointers({x, weight, bias, grad_out, dx, initial_state, grad_final_state, grad_initial_state}, lengths)) != LA_OK)
        return st;
    if (!aligned(dweight, 4) || (dbias && !aligned(dbias, 4))) return LA_ERR_ALIGN;
    ConvParams p{};
    if ((st = strides_of(x_strides, B, N, E, dtype, &p.sx)) != LA_OK) return st;
    if ((st = strides_of(g_strides, B, N, E, dtype, &p.sg)) != LA_OK) return st;
    if (!workspace || ws_bytes < la_conv_workspace_size(B, N, E, W, dtype)) return LA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return LA_ERR_ALIGN;
    p.x = x; p.weight = weight; p.bias = bias; p.g = grad_out; p.out = dx; p.dweight = dweight; p.dbias = dbias;
    p.init = initial_state; p.dfinal = grad_final_state; p.dinit = grad_initial_state; p.lengths = lengths;
    p.part = static_cast<float *>(workspace);
    p.B = B; p.N = N; p.E = E; p.silu = silu; p.wide = weight_dtype == LA_F32;
    p.run = grad_run(B, N, E);
    p.runs = (N + p.run - 1) / p.run;
    p.parts = grad_parts(B, N, E);
    if ((long long)((E + 127) / 128) * p.parts >= (1ll << 31) - 1) return LA_ERR_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = dtype == LA_BF16 ? gradient<__nv_bfloat16>(p, W, s) : gradient<float>(p, W, s);
    return e == cudaSuccess ? LA_OK : cuda_fail(e);
}

la_status la_conv_step(const void *x, const void *weight, const void *bias, void *out, const void *state, void *state_out,
                       const int *slots, int pool, int B, int E, int W, la_dtype dtype, la_dtype weight_dtype, int silu,
                       const la_strides *x_strides, void *stream) {
    la_status st = check(B, 1, E, W, dtype, weight_dtype);
    if (st != LA_OK) return st;
    if (!x || !weight || !out || !state || !state_out || pool <= 0 || (!slots && pool < B)) return LA_ERR_ARG;
    if ((st = bad_pointers({x, weight, bias, out, state, state_out}, slots)) != LA_OK) return st;
    ConvParams p{};
    if ((st = strides_of(x_strides, B, 1, E, dtype, &p.sx)) != LA_OK) return st;
    p.x = x; p.weight = weight; p.bias = bias; p.out = out; p.init = state; p.fin = state_out; p.slots = slots;
    p.pool = pool; p.B = B; p.N = 1; p.E = E; p.silu = silu; p.wide = weight_dtype == LA_F32;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = dtype == LA_BF16 ? step<__nv_bfloat16>(p, W, s) : step<float>(p, W, s);
    return e == cudaSuccess ? LA_OK : cuda_fail(e);
}

}  // extern "C"
