// la_decay.cuh -- shared definitions of the decayed linear attention (la_decay_*).
//
// All the chunked products have one form, a pass F(X, Y, Z) over the tokens in order:
//
//   F_i = sum_{j <= i} gamma^(i-j) (x_i . y_j) z_j + gamma^(i+1) x_i^T S_0
//
// forward:  out = F(q, k, v), S = sum k v^T;
// backward: dq = F(g, v, k) with S^T; and, with the tokens in reverse order and
// A = sum q g^T in the place of S, dv = F(k, q, g) with A and dk = F(v, g, q) with A^T, summed over
// the query heads of each group.  (A_i = sum_{j >= i} gamma^(j-i) q_j g_j^T is the gradient of S_i.)
#pragma once

#include "la_internal.cuh"

namespace la {

// A pass.  Tokens are counted along its direction (`rev`: from the last to the first).
struct DecayPass {
    const void *x, *y, *z;      // [B, Hx, N, DX], [B, Hyz, N, DX], [B, Hyz, N, DZ]
    Strides sx, sy, sz;
    void *out;                  // [B, Hx, N, DZ], contiguous
    const float *slots;         // nseg > 1: workspace.  CUDA cores: [B Hkv][nseg] states [D][Dv], slot 0 the
                                // starting state, slot u > 0 the sum over segment u - 1 alone.  Tensor cores:
                                // [B Hkv][nseg] starting states of the segments, lane-blocked (decay_blocked) in the
                                // pass's own orientation
    const float *init;          // nseg = 1: starting state [B Hkv][D][Dv] or null
    float *fin;                 // CUDA cores: state after the last token, or null
    int tr;                     // the pass's DX x DZ state is the transpose of the stored D x Dv one
    int many_yz;                // Hyz = n_rep Hkv heads of y and z for each head of x (summed into one
                                // out); else Hx = n_rep Hkv heads of x for each head of y and z
    int rev;
    // reverse order: the incoming gradient of the last state has not decayed when it meets the first
    // token of the pass, so its powers of gamma are one lower (first_off = 1), and what
    // leaves at the other end decays once more
    int first_off;
    float init_mul, fin_mul;    // the reverse states leave out `scale`, which comes in and goes out here
};

struct DecayParams {
    const float *log_decay;     // [Hkv]
    const int *lengths;         // [B] or null
    int B, Hkv, n_rep, N, D, Dv;
    float scale;
    int seg_len, nseg;
    int npass;
    DecayPass pass[3];
    int *err;
};

// The sums over single segments that later segments start from: for segment u, the sum of
// gamma^(tokens after j in the segment) y_j z_j^T (over the heads of y, z), a state D x Dv.
// CUDA cores: in slot u + 1, [D][Dv], with the starting state (times init_mul) in slot 0.
// Tensor cores: the first nsum segments in nsub parts each (more blocks than segments: the kernel is short), in
// part[nsum nsub], lane-blocked; decay_tc_join() then makes the segments' starting states of them.
struct DecayStateParams {
    const float *log_decay;
    const int *lengths;
    const void *y[2], *z[2];
    Strides sy[2], sz[2];
    const float *init[2];
    float init_mul[2];
    int heads[2];               // heads of y and z per key/value head
    int rev[2];
    float *slots[2];
    int exact[2];               // a float32 state that the caller gets depends on these sums (tensor cores)
    float *fin[2];              // tensor cores: the state after the last segment, or null (its sum is taken
    float fin_mul[2];           // too then: nsum = nseg segments)
    int direct;                 // tensor cores: one part in all, the state kernel writes fin itself
    int nsum;
    int first, n;               // state arrays of this launch: [first, first + n)
    int B, Hkv, N, D, Dv, seg_len, nseg;
    int nsub, sub_len;          // tensor cores: parts of a segment
    float *part[2];
    float *start[2], *start_tr[2];   // ... and where the starting states go: as S, and as its transpose (or null)
    int first_off[2];
    int *err;
};

// Lane-blocked states: element (row d, column e) of R rows at ((e / 4) R + d) 4 + e % 4, so that a warp whose
// threads hold rows moves 16 bytes of each in one run.
__host__ __device__ constexpr size_t decay_blocked(int R, int d, int e) { return ((size_t)(e / 4) * R + d) * 4 + e % 4; }

// Tokens of sequence b.
__device__ __forceinline__ int decay_tokens(const int *lengths, int b, int N) {
    return lengths ? min(max(lengths[b], 0), N) : N;
}

// log2(gamma) of a head, with -inf (gamma = 0) kept finite so that gamma^0 = 2^(0 x) stays 1: 2^-1e30
// and every power of it is 0.
__device__ __forceinline__ float decay_log2(float log_decay) {
    const float l2 = log_decay * 1.4426950408889634f;
    return l2 < -1e30f ? -1e30f : l2;
}

// CUDA-core kernels (la_decay_simt.cu): every dtype, width and stride.
inline int decay_simt_slice(int DZ) { return DZ < 64 ? DZ : 64; }   // columns of out that a block owns
cudaError_t decay_simt_states(const DecayStateParams &p, la_dtype dt, cudaStream_t s);
cudaError_t decay_simt_passes(const DecayParams &p, int pass0, int npass, la_dtype dt, cudaStream_t s);

// Tensor-core kernels (la_decay_tc.cu): bfloat16, widths 64 and 128.  Segments are cut in token
// order, multiples of kDecayTcChunk tokens; every pass of a call in one launch where the widths allow.
constexpr int kDecayTcChunk = 128;
cudaError_t decay_tc_states(const DecayStateParams &p, cudaStream_t s);
cudaError_t decay_tc_join(const DecayStateParams &p, cudaStream_t s);
cudaError_t decay_tc_passes(const DecayParams &p, cudaStream_t s);

// One token (la_decay_step).
struct DecayStepParams {
    const void *q, *k, *v;
    Strides sq, sk, sv;
    void *out;
    const float *state;
    float *state_out;
    const float *log_decay;
    const int *slots;
    int pool, B, Hkv, n_rep, D, Dv;
    float scale;
};
cudaError_t decay_step(const DecayStepParams &p, la_dtype dt, cudaStream_t s);

}  // namespace la
