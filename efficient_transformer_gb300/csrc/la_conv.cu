// la_conv.cu -- short causal convolution of every channel with W taps, with silu or without: forward, gradient, single
// token, and their C ABI.
//
//   v_t = bias + sum_j w_j x_(t - W + 1 + j),   out_t = v_t sigmoid(v_t)
//   g'_t = g_t (v sigmoid(v))',   dx_t = sum_j w_j g'_(t + W - 1 - j),   dw_j = sum_t g'_t x_(t - W + 1 + j),   db = sum g'
//
// Bound by memory: each row is read once but for the W - 1 rows at a run's edge.  A thread owns four channels (one load a
// token) and walks a run of tokens with the last W rows in registers, two channels an instruction; the next tokens' loads
// are issued before the present ones are worked on.  65536 x 2048 bfloat16: 86 us, 6.2 TB/s; the gradient of 4 x 4096 x 4096 85 us,
// 4.7 TB/s (128 registers, 16 warps an SM).  float32: 167 us, 6.4 TB/s, and 211 us, 3.8 TB/s (the bound of 128 registers, chosen for
// bfloat16, spills 388 bytes there).
#include <climits>
#include <initializer_list>
#include <type_traits>

#include "la_ssm.cuh"

namespace la {
namespace {

struct ConvParams {
    const void *x, *g, *weight, *bias, *init, *dfinal;
    Strides sx, sg;
    const int *lengths, *slots;
    void *out, *fin, *dinit, *dweight, *dbias;
    float *part;                  // gradient: [parts][W + 1][E]
    int B, N, E, silu, wide;      // wide: weight and bias are float32
    int run, runs, parts, pool;
};

constexpr int kV = 4;             // channels of a thread: 8 bytes of bfloat16, 16 of float32, a token

// kV channels of a row, as they lie: widened where they are used, so that a load's wait is there and not at a copy
template <typename T>
struct Row;
template <>
struct __align__(8) Row<__nv_bfloat16> {
    unsigned v[2];
};
template <>
struct __align__(16) Row<float> {
    float v[4];
};
template <typename T>
__device__ __forceinline__ Row<T> no_row() {
    Row<T> r;
#pragma unroll
    for (auto &x : r.v) x = 0;
    return r;
}
template <typename T>
__device__ __forceinline__ Row<T> get_row(const void *base, long long at) {
    return *reinterpret_cast<const Row<T> *>(static_cast<const T *>(base) + at);
}
template <typename T>
__device__ __forceinline__ void put_row(void *base, long long at, const Row<T> &r) {
    *reinterpret_cast<Row<T> *>(static_cast<T *>(base) + at) = r;
}
__device__ __forceinline__ F2 pair(const Row<__nv_bfloat16> &r, int c) {
    return F2{__uint_as_float(r.v[c] << 16), __uint_as_float(r.v[c] & 0xffff0000u)};
}
__device__ __forceinline__ F2 pair(const Row<float> &r, int c) { return F2{r.v[2 * c], r.v[2 * c + 1]}; }
__device__ __forceinline__ void set(Row<__nv_bfloat16> &r, F2 a, F2 b) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r.v[0]) : "f"(a.y), "f"(a.x));
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r.v[1]) : "f"(b.y), "f"(b.x));
}
__device__ __forceinline__ void set(Row<float> &r, F2 a, F2 b) {
    r.v[0] = a.x;
    r.v[1] = a.y;
    r.v[2] = b.x;
    r.v[3] = b.y;
}
template <typename T>
__device__ __forceinline__ Row<T> row_of(F2 a, F2 b) {
    Row<T> r;
    set(r, a, b);
    return r;
}

// A thread's weights, two channels a pair, and its bias; float32 or T, as they lie.
template <typename T, int W>
struct Taps {
    F2 w[W][2], bias[2];
    __device__ __forceinline__ Taps(const ConvParams &p, int e) {
        float f[kV * W];
#pragma unroll
        for (int q = 0; q < W; ++q) {
            if (p.wide) take(f + kV * q, get_row<float>(p.weight, (long long)e * W + kV * q));
            else take(f + kV * q, get_row<T>(p.weight, (long long)e * W + kV * q));
        }
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int c = 0; c < 2; ++c) w[j][c] = F2{f[2 * c * W + j], f[(2 * c + 1) * W + j]};
        float g[kV] = {0.f, 0.f, 0.f, 0.f};
        if (p.bias) {
            if (p.wide) take(g, get_row<float>(p.bias, e));
            else take(g, get_row<T>(p.bias, e));
        }
        bias[0] = F2{g[0], g[1]};
        bias[1] = F2{g[2], g[3]};
    }
    template <typename U>
    static __device__ __forceinline__ void take(float *to, const Row<U> &r) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const F2 f = pair(r, c);
            to[2 * c] = f.x;
            to[2 * c + 1] = f.y;
        }
    }
};

// Row t of a sequence with the W - 1 inputs before its first token (`len` tokens; past them: zeros).
template <typename T, int W>
struct Source {
    const void *x, *init;
    long long x0, s0, step, E;
    int len;
    __device__ __forceinline__ Source(const ConvParams &p, int b, int e, int len)
        : x(p.x), init(p.init), x0(b * p.sx.b + e), s0((long long)b * (W - 1) * p.E + e), step(p.sx.n), E(p.E), len(len) {}
    __device__ __forceinline__ Row<T> operator()(int t) const {
        if (t >= 0) return t < len ? get_row<T>(x, x0 + t * step) : no_row<T>();
        return init ? get_row<T>(init, s0 + (t + W - 1) * E) : no_row<T>();
    }
};

// Q rows from token t on (their pointer at hand: it moves on); all of them within the length, or one by one.
template <typename T, int Q, typename F>
__device__ __forceinline__ void ask(Row<T> (&to)[Q], const T *&at, long long step, bool whole, F one) {
    if (whole) {
#pragma unroll
        for (int q = 0; q < Q; ++q) to[q] = get_row<T>(at, q * step);
    } else {
#pragma unroll
        for (int q = 0; q < Q; ++q) to[q] = one(q);
    }
    at += Q * step;
}

constexpr int kBatch = 8;         // tokens whose loads are issued together

// Forward.  Thread: four channels, `run` tokens (a multiple of kBatch) of one sequence.
template <typename T, int W>
__global__ void __launch_bounds__(256, 2) k_conv(ConvParams p) {
    pdl_wait();
    const int vecs = p.E / kV;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= (long long)p.B * p.runs * vecs) return;
    const int e = (int)(i % vecs) * kV, run = (int)(i / vecs % p.runs), b = (int)(i / vecs / p.runs);
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.N) : p.N;
    const int t0 = run * p.run, t1 = min(t0 + p.run, p.N);
    const Source<T, W> row(p, b, e, len);
    Row<T> in[kBatch], next[kBatch];
    const T *at = static_cast<const T *>(p.x) + row.x0 + t0 * row.step;
    const int te = min(t1, len);
    ask<T>(next, at, row.step, t0 + kBatch <= te, [&](int q) { return row(t0 + q); });
    F2 win[W][2];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const Row<T> r = row(t0 - (W - 1) + j);
        win[j + 1][0] = pair(r, 0);
        win[j + 1][1] = pair(r, 1);
    }
    const Taps<T, W> k(p, e);
    // The first run's thread alone reads the initial state; having read it, it writes the final one, which may take its place.
    if (run == 0 && p.fin) {
        Row<T> last[W - 1];
#pragma unroll
        for (int j = 0; j < W - 1; ++j) last[j] = row(len - (W - 1) + j);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) put_row<T>(p.fin, row.s0 + (long long)j * p.E, last[j]);
    }
    T *out = static_cast<T *>(p.out) + ((long long)b * p.N + t0) * p.E + e;
    for (int t = t0; t < t1; t += kBatch) {
#pragma unroll
        for (int q = 0; q < kBatch; ++q) in[q] = next[q];
        if (t + kBatch < te) ask<T>(next, at, row.step, t + 2 * kBatch <= te, [&](int q) { return row(t + kBatch + q); });
        auto each = [&](auto whole) {   // (whole: all of these tokens are within the length and the run)
#pragma unroll
            for (int q = 0; q < kBatch; ++q) {
                F2 v[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) win[j][c] = win[j + 1][c];
                    win[W - 1][c] = pair(in[q], c);
                    v[c] = k.bias[c];
#pragma unroll
                    for (int j = 0; j < W; ++j) v[c] = fma2(k.w[j][c], win[j][c], v[c]);
                    if (p.silu) v[c] = mul2(v[c], sigmoid(v[c]));
                }
                if (whole.value) put_row<T>(out, (long long)q * p.E, row_of<T>(v[0], v[1]));
                else if (t + q < t1) put_row<T>(out, (long long)q * p.E, t + q < len ? row_of<T>(v[0], v[1]) : no_row<T>());
            }
        };
        if (t + kBatch <= te) each(std::true_type{});
        else each(std::false_type{});
        out += (long long)kBatch * p.E;
    }
}

// Gradient.  Block: 32 x 4 channels, 8 runs of one sequence; dw and db of a thread's run are added up over the block.
template <typename T, int W>
__global__ void __launch_bounds__(256, 2) k_conv_grad(ConvParams p) {
    constexpr int Q = 4;
    __shared__ float sums[8][W + 1][32 * kV];
    pdl_wait();
    const int tiles = (p.E + 32 * kV - 1) / (32 * kV), groups = (p.runs + 7) / 8;
    const int tile = blockIdx.x % tiles, grp = blockIdx.x / tiles % groups, b = blockIdx.x / tiles / groups;
    const int lane = threadIdx.x % 32, y = threadIdx.x / 32, e = (tile * 32 + lane) * kV, run = grp * 8 + y;
    const int len = p.lengths ? min(max(p.lengths[b], 0), p.N) : p.N;
    const int t0 = run * p.run, t1 = min(t0 + p.run, p.N);
    F2 dw[W][2], db[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        db[c] = f2(0.f);
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][c] = f2(0.f);
    }
    if (e < p.E && t0 < p.N) {
        const Source<T, W> row(p, b, e, len);
        const long long g0 = b * p.sg.b + e;
        auto grad = [&](int t) { return t < len ? get_row<T>(p.g, g0 + t * p.sg.n) : no_row<T>(); };
        Row<T> in[Q], gin[Q], next[Q], gnext[Q];
        const T *xat = static_cast<const T *>(p.x) + row.x0 + t0 * row.step, *gat = static_cast<const T *>(p.g) + g0 + t0 * p.sg.n;
        const int tw = min(t1 + W - 1, len);   // (of the rows past the run only what is within the length)
        ask<T>(next, xat, row.step, t0 + Q <= tw, [&](int q) { return row(t0 + q); });
        ask<T>(gnext, gat, p.sg.n, t0 + Q <= tw, [&](int q) { return grad(t0 + q); });
        F2 win[W][2], gw[W][2];   // rows x_(t - W + 1 ..  t) and g'_(t - W + 1 .. t)
#pragma unroll
        for (int j = 0; j < W; ++j) gw[j][0] = gw[j][1] = f2(0.f);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            const Row<T> r = row(t0 - (W - 1) + j);
            win[j + 1][0] = pair(r, 0);
            win[j + 1][1] = pair(r, 1);
        }
        const Taps<T, W> k(p, e);
        T *dx = static_cast<T *>(p.out) + (long long)b * p.N * p.E + e;
        // token t gives g'_t and with it the gradient of row t - W + 1; the first run starts with the rows before the first
        // token, the others end W - 1 tokens past their run
        for (int t = t0; t < t1 + W - 1; t += Q) {
#pragma unroll
            for (int q = 0; q < Q; ++q) {
                in[q] = next[q];
                gin[q] = gnext[q];
            }
            if (t + Q < t1 + W - 1) {
                ask<T>(next, xat, row.step, t + 2 * Q <= tw, [&](int q) { return row(t + Q + q); });
                ask<T>(gnext, gat, p.sg.n, t + 2 * Q <= tw, [&](int q) { return grad(t + Q + q); });
            }
            auto each = [&](auto whole) {   // (whole: all of these tokens are within the length and the run, their rows too)
#pragma unroll
                for (int q = 0; q < Q; ++q) {
                    const int at = t + q - (W - 1);   // the row whose gradient is whole now
                    F2 d[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
#pragma unroll
                        for (int j = 0; j < W - 1; ++j) {
                            win[j][c] = win[j + 1][c];
                            gw[j][c] = gw[j + 1][c];
                        }
                        win[W - 1][c] = pair(in[q], c);
                        F2 g = pair(gin[q], c);
                        if (p.silu) {
                            F2 v = k.bias[c];
#pragma unroll
                            for (int j = 0; j < W; ++j) v = fma2(k.w[j][c], win[j][c], v);
                            // (v sigmoid(v))' = s + v s (1 - s)
                            const F2 s = sigmoid(v), vs = mul2(v, s);
                            g = mul2(g, add2(s, fma2(F2{-vs.x, -vs.y}, s, vs)));
                            if (!whole.value && t + q >= len) g = f2(0.f);
                        }
                        gw[W - 1][c] = g;
                        if (whole.value || (t + q < t1 && t + q < len)) {   // (past the length g' = 0, but the window need not be finite)
                            db[c] = add2(db[c], g);
#pragma unroll
                            for (int j = 0; j < W; ++j) dw[j][c] = fma2(g, win[j][c], dw[j][c]);
                        }
                        d[c] = mul2(k.w[0][c], gw[W - 1][c]);
#pragma unroll
                        for (int j = 1; j < W; ++j) d[c] = fma2(k.w[j][c], gw[W - 1 - j][c], d[c]);
                    }
                    if (whole.value) {
                        put_row<T>(dx, (long long)at * p.E, row_of<T>(d[0], d[1]));
                        continue;
                    }
                    // (a thread's first W - 1 rows are whole in the run before, but for those in front of the first token)
                    const bool front = at < 0;
                    if (at >= t1 || (front ? run != 0 || !p.dinit : at < t0)) continue;
                    const int f = at + (W - 1) - len;   // the row's place in the final state
                    if (p.dfinal && f >= 0 && f < W - 1) {
                        const Row<T> add = get_row<T>(p.dfinal, row.s0 + (long long)f * p.E);
                        d[0] = add2(d[0], pair(add, 0));
                        d[1] = add2(d[1], pair(add, 1));
                    }
                    const Row<T> o = at < len ? row_of<T>(d[0], d[1]) : no_row<T>();
                    if (front) put_row<T>(p.dinit, row.s0 + (long long)(at + W - 1) * p.E, o);
                    else put_row<T>(dx, (long long)at * p.E, o);
                }
            };
            if (t >= t0 + W - 1 && t + Q <= min(t1, len)) each(std::true_type{});
            else each(std::false_type{});
        }
    }
#pragma unroll
    for (int j = 0; j <= W; ++j)
        *reinterpret_cast<float4 *>(&sums[y][j][lane * kV]) =
            j < W ? make_float4(dw[j < W ? j : 0][0].x, dw[j < W ? j : 0][0].y, dw[j < W ? j : 0][1].x, dw[j < W ? j : 0][1].y)
                  : make_float4(db[0].x, db[0].y, db[1].x, db[1].y);
    __syncthreads();
    float *part = p.part + (size_t)(b * groups + grp) * (W + 1) * p.E;
    for (int i = threadIdx.x; i < (W + 1) * 32 * kV; i += 256) {
        const int j = i / (32 * kV), c = i % (32 * kV);
        float s = 0.f;
#pragma unroll
        for (int q = 0; q < 8; ++q) s += sums[q][j][c];
        if (tile * 32 * kV + c < p.E) part[(size_t)j * p.E + tile * 32 * kV + c] = s;
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
    pdl_wait();
    const int vecs = p.E / kV;
    const long long i = (long long)blockIdx.x * 128 + threadIdx.x;
    if (i >= (long long)p.B * vecs) return;
    const int e = (int)(i % vecs) * kV, b = (int)(i / vecs);
    const int slot = p.slots ? p.slots[b] : b;
    const Row<T> x = get_row<T>(p.x, b * p.sx.b + e);
    const Taps<T, W> k(p, e);
    if (slot < 0 || slot >= p.pool) {
        put_row<T>(p.out, (long long)b * p.E + e, no_row<T>());
        return;
    }
    const long long s0 = (long long)slot * (W - 1) * p.E + e;
    Row<T> win[W];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j] = get_row<T>(p.init, s0 + (long long)j * p.E);
    win[W - 1] = x;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) put_row<T>(p.fin, s0 + (long long)j * p.E, win[j + 1]);
    F2 v[2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        v[c] = k.bias[c];
#pragma unroll
        for (int j = 0; j < W; ++j) v[c] = fma2(k.w[j][c], pair(win[j], c), v[c]);
        if (p.silu) v[c] = mul2(v[c], sigmoid(v[c]));
    }
    put_row<T>(p.out, (long long)b * p.E + e, row_of<T>(v[0], v[1]));
}

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Sizes and types; the weight's type is float32 or the inputs'.
la_status check(int B, int N, int E, int W, la_dtype dt, la_dtype wt) {
    if (B <= 0 || N <= 0 || E <= 0 || (dt != LA_F32 && dt != LA_BF16) || (wt != LA_F32 && wt != dt)) return LA_ERR_ARG;
    if (E > INT_MAX - 127) return LA_ERR_ARG;   // (the end of the last tile of 128 channels)
    if (N > (1 << 30) || (long long)B * N > (1ll << 40) || (long long)B * E > (1ll << 39)) return LA_ERR_ARG;
    if (W < 2 || W > 4 || E % 8) return LA_ERR_UNSUPPORTED;
    return LA_OK;
}

// Tokens of a thread's run (a multiple of `unit`): a run costs its tokens and about `start` more (the rows before it, the
// weights, the first loads' latency), and the grid takes whole waves of two blocks an SM.
template <typename F>
int best_run(int N, int unit, int start, F blocks) {
    int best = unit;
    double least = -1.0;
    for (int run = unit; run <= 256 && run < N + unit; run += unit) {
        const long long waves = (blocks((N + run - 1) / run) + 2 * kPlanSms - 1) / (2 * kPlanSms);
        const double cost = (double)waves * (run + start);
        if (least < 0 || cost < least) {
            least = cost;
            best = run;
        }
    }
    return best;
}
int forward_run(int B, int N, int E) {
    return best_run(N, kBatch, 16, [&](long long runs) { return (B * runs * (E / kV) + 255) / 256; });
}
int grad_run(int B, int N, int E) {
    return best_run(N, 4, 16, [&](long long runs) { return (E + 127) / 128 * ((runs + 7) / 8) * B; });
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
    const long long threads = (long long)p.B * p.runs * (p.E / kV);
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
    const long long threads = (long long)p.B * (p.E / kV);
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
    p.run = forward_run(B, N, E);
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
