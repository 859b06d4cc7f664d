// Internal interface of the first-order linear attention with a decay for each head
// (linattn_api.cu composes the passes; linattn_simt.cu and linattn_tc.cu run them).
//
// Every pass is the same scan over rows t of one state head, forward or in reverse:
//     y_t = s_fin (s_col sum_i g^|t-i| (x_t . k_i) v_i + g^(distance to the carry) x_t^T Sig)
// over the valid rows i <= t (reverse: i >= t) of t's segment, Sig (dx x dy, float32) being the
// state that enters the segment:  forward  Sig = sum_i g^(t0-1-i) k_i v_i^T  (the state
// before the segment's first row t0),  reverse  Sig = sum_i g^(i-t1) k_i v_i^T  (t1 the row
// after the segment's last).  With
//     forward output   x = q,    k = k,    v = v
//     dq               x = dout, k = v,    v = k     (Sig: the forward states, transposed)
//     dv  (reverse)    x = k,    k = q,    v = dout
//     dk  (reverse)    x = v,    k = dout, v = q     (Sig: the reverse states, transposed)
#pragma once

#include "common.cuh"

namespace hla2 {

struct LinPass {
    hla2_view x, k, v;
    hla2_view y;               // written
    int B, Hs;                 // state heads: grid rows are b * Hs + s
    int rx, rk;                // x / y heads s rx .. and key / value heads s rk .. per state head; one of them is 1
    int n, dx, dy;
    int W, nchunks, seg_chunks, nseg;
    int rev;
    float s_col, s_fin, s_state;  // s_state: factor of k v^T in the state
    const float* gamma;        // [Hs] or NULL
    const int* lengths;        // [B] or NULL
    const float* carry;        // [B Hs][nseg] states entering the segments, or NULL (zero)
    int carry_t;               // they are stored dy x dx
    // Tensor-core output pass, in place of carry and with the meaning that launch_lin_scan gives them: the
    // segments' sums, the state before the scan, and where the one after it goes.  Each may be NULL.
    const float *prior, *init;
    float* fin;
    int exact_sums;            // the sums end in a state that is returned: exact to float32
    float* sums;               // summary pass: [B Hs][nseg][dx dy], each segment's state from zero
    int* status;               // word that a wait which gave up is recorded in
};

__host__ __device__ inline int lin_len(const int* lengths, int b, int n) {
    if (!lengths) return n;
    const int l = lengths[b];
    return l < 0 ? 0 : l > n ? n : l;
}

// Valid rows of the first i segments in the scan's direction
__device__ __forceinline__ int lin_rows_before(int len, int rev, int i, int nseg, int seg_rows) {
    return rev ? len - (int)min((long long)len, (long long)(nseg - i) * seg_rows)
               : (int)min((long long)len, (long long)i * seg_rows);
}

__device__ __forceinline__ float lin_decay(const LinPass& a, int s) { return a.gamma ? __ldg(a.gamma + s) : 1.0f; }

// Every kernel here is launched so that it may start while the one before it on the stream drains
// (launch_pdl): it sets itself up, then waits (pdl_wait) before it touches global memory.

// SIMT passes (float32, any size); W = lin_simt_width(dx, dy, state heads, n, SMs):
// 64 rows (32 where a dimension is 128, for the shared memory), and half or a quarter of that while the
// chunks of all heads would not give every SM one.  Two heads of 1023 rows, d = 32, dv = 64: the output
// pass took 31 us with 64 rows a chunk (32 CTAs), 12 us with 16 (128 CTAs).
int lin_simt_width(int dx, int dy, long long heads, int n, int sms);
int lin_simt_ctas(int dx, int dy, int W);  // resident CTAs per SM
// Passes of one call that do not wait for each other go in one launch where they are small: the training step of
// 2 heads of 1023 rows took 67 us in ten launches and takes 49 us in six.
constexpr int kLinPasses = 3;
struct LinPasses {
    LinPass p[kLinPasses];
};
int launch_lin_simt(const LinPass* passes, int count, bool summary, cudaStream_t st);

// Tensor-core passes (bf16, any size; linattn_tc.cu): W = 128, one CTA per SM.  Its output pass
// can join the segments' sums itself.
int launch_lin_tc(const LinPass& a, bool summary, cudaStream_t st);

// States entering the segments from the segment summaries, for each state element:
// carry[s] = cur;  cur = g^(valid rows of s) cur + sums[s]  in the scan's direction.  init (nullable) is the state before the scan; reverse: the gradient of the
// final state, which enters as init / g.  final (nullable) receives the state after it;
// reverse: times g, the gradient of the initial state.  sums may be NULL with nseg == 1 and no final.
// `count` scans (1 or 2) of the same sizes in one launch.
struct LinScan {
    const float* sums;
    float* carry;
    const float* init;
    float* final_state;
    int rev;
};
int launch_lin_scan(const LinScan* scans, int count, const float* gamma, const int* lengths, int B, int Hs, int n,
                    int seg_rows, int nseg, int elems, cudaStream_t st);

int launch_lin_step(float* state, const void* q, const void* k, const void* v, void* out, int N, int H, int Hk, int d,
                    int dv, const float* gamma, float scale, bool is_bf16, cudaStream_t st);

}  // namespace hla2
