// Causal linear attention with a decay for each head, g = exp(log_decay_h):
//     S_t = g S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t,
// from a state S_0 to a state S_n (d x d, fp32), its form for one token, and
// its gradients.  With G the gradient of the state after a token,
//     G_t = g G_{t+1} + scale q_t dout_t^T  (g G_{n+1} replaced by dS_n),
//     dq_t = scale S_t dout_t,  dk_t = G_t v_t,  dv_t = G_t^T k_t,  dS_0 = g G_1,
// so each gradient is the same operator again: dq that of (dout, v, k) from
// the transposed state, dk and dv those of (v, dout, q) and (k, q, dout) run
// from the last token to the first.
//
// Method: the chunk-wise form of "Gated Linear Attention Transformers with
// Hardware-Efficient Training" (nubint.ai review) and the intra-/inter-block
// split of "Lightning Attention-2" (chatpaper.ai summary), with that paper's
// decay.
#pragma once

#include "ptx.cuh"

namespace attn {

// One pass of the operator over x_t (in place of q), y_t (k) and z_t (v).
struct DecayPass {
    const void* x;
    const void* y;
    const void* z;
    void* out;
    const float* init;   // (B, H, D, D) or null: the state before the first token
    float* last;         // (B, H, D, D) or null: the state after the last token
    int transposed;      // init is stored transposed
    int reverse;         // tokens are walked from the last to the first
};

struct DecayParams {
    DecayPass pass[3];
    const float* log_decay;  // (H)
    const int* lens;         // (B) or null
    int B, H, N;
    float scale;
};

__device__ __forceinline__ int decay_len(const int* lens, int b, int N) {
    if (!lens) return N;
    const int n = lens[b];
    return n < 0 ? 0 : (n > N ? N : n);
}

// log_decay -inf (no memory at all) times 0 would not be 0: held at -1e4,
// whose exponential is 0.
__device__ __forceinline__ float decay_log(const float* log_decay, int h) {
    return fmaxf(log_decay[h], -1e4f);
}

// Token by token: one CTA per (pass, head), thread = column of the state.
template <int D, bool BF16>
__global__ void __launch_bounds__(D) decay_recurrent_kernel(const DecayParams p) {
    __shared__ float sx[D], sy[D];
    const int bh = blockIdx.x, h = bh % p.H, b = bh / p.H, c = threadIdx.x;
    const DecayPass& ps = p.pass[blockIdx.y];
    const int n = decay_len(p.lens, b, p.N);
    const float g = expf(decay_log(p.log_decay, h));
    const size_t state = static_cast<size_t>(bh) * D * D;
    // backwards the state is a gradient: scale enters with each token's term
    // instead of with the result, and the decay follows the token
    const float in = ps.reverse ? p.scale : 1.f, out = ps.reverse ? 1.f : p.scale;
    float S[D];
#pragma unroll
    for (int a = 0; a < D; ++a)
        S[a] = ps.init ? ps.init[state + (ps.transposed ? c * D + a : a * D + c)] : 0.f;
    auto at = [&](const void* m, int t) {
        const uint16_t v = static_cast<const uint16_t*>(m)[(static_cast<size_t>(bh) * p.N + t) * D + c];
        const float2 f = unpack2<BF16>(v);
        return f.x;
    };
    for (int i = 0; i < n; ++i) {
        const int t = ps.reverse ? n - 1 - i : i;
        __syncthreads();
        sx[c] = at(ps.x, t);
        sy[c] = at(ps.y, t);
        const float z = at(ps.z, t) * in;
        __syncthreads();
        float o = 0.f;
#pragma unroll
        for (int a = 0; a < D; ++a) {
            const float s = (ps.reverse ? S[a] : g * S[a]) + sy[a] * z;
            o += sx[a] * s;
            S[a] = ps.reverse ? g * s : s;
        }
        static_cast<uint16_t*>(ps.out)[(static_cast<size_t>(bh) * p.N + t) * D + c] =
            static_cast<uint16_t>(pack2<BF16>(o * out, 0.f));
    }
    if (ps.last) {
#pragma unroll
        for (int a = 0; a < D; ++a)
            ps.last[state + a * D + c] = S[a];
    }
}

// One token: one CTA per head, thread = column of the state.
template <int D, bool BF16>
__global__ void __launch_bounds__(D) decay_step_kernel(const void* q, const void* k, const void* v,
                                                       const float* log_decay, const float* in,
                                                       float* out, void* o, int H, float scale) {
    __shared__ float sq[D], sk[D];
    const int bh = blockIdx.x, c = threadIdx.x;
    auto at = [&](const void* m) {
        return unpack2<BF16>(static_cast<const uint16_t*>(m)[static_cast<size_t>(bh) * D + c]).x;
    };
    sq[c] = at(q);
    sk[c] = at(k);
    const float z = at(v), g = expf(decay_log(log_decay, bh % H));
    __syncthreads();
    const size_t state = static_cast<size_t>(bh) * D * D;
    float acc = 0.f;
#pragma unroll 8
    for (int a = 0; a < D; ++a) {
        const float s = g * in[state + a * D + c] + sk[a] * z;
        acc += sq[a] * s;
        out[state + a * D + c] = s;
    }
    static_cast<uint16_t*>(o)[static_cast<size_t>(bh) * D + c] =
        static_cast<uint16_t>(pack2<BF16>(acc * scale, 0.f));
}

}  // namespace attn
