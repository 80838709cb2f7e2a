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

#include "ptx_more.cuh"

namespace attn {

// One pass of the operator over x_t (in place of q), y_t (k) and z_t (v).
struct DecayPass {
    int x, y, z;         // which of the tensor maps
    int out_map;         // and the result's
    void* out;           // (B, H, N, D)
    const float* init;   // (B, H, D, D) or null: the state before the first token
    float* last;         // (B, H, D, D) or null: the state after the last token
    int transposed;      // init is stored transposed
    int reverse;         // tokens are walked from the last to the first
};

struct DecayParams {
    DecayPass pass[3];
    const float* log_decay;  // (H)
    const int* lens;         // (B) or null
    float* seg;              // (passes, nseg, B H, D, D): states of the segments
    int passes, B, H, N;
    int nseg, seg_chunks;    // a sequence's chunks in segments of seg_chunks
    int zero_past;           // the result's rows past a sequence's end: zeros, else untouched
    float scale;
};

struct DecayMaps {
    CUtensorMap m[7];
};

__device__ __forceinline__ int decay_len(const int* lens, int b, int N) {
    if (!lens) return N;
    const int n = lens[b];
    return n < 0 ? 0 : (n > N ? N : n);
}

// log_decay -inf (no memory at all) times 0 would not be 0: held at -1e4,
// whose exponential is 0.
__device__ __forceinline__ float decay_log(const float* log_decay, int h) {
    const float x = log_decay[h];
    return x < -1e4f ? -1e4f : x;  // NaN stays
}

// The power of two that brings values of largest magnitude `top` to 2^14 .. 2^15, where
// fp16 holds all that is above 2^-29 of it as normal numbers (1 for 0 and NaN); its
// inverse is a normal number too.
__device__ __forceinline__ float fp16_up(float top) {
    const int e = top > 0.f ? 268 - static_cast<int>(__float_as_uint(top) >> 23) : 127;
    return __uint_as_float(static_cast<uint32_t>(e < 1 ? 1 : (e > 253 ? 253 : e)) << 23);
}

// The inverse of a power of two that fp16_up gives.
__device__ __forceinline__ float fp16_down(float up) { return __uint_as_float((254u << 23) - __float_as_uint(up)); }

constexpr int kDecayChunk = 128;

// Tokens of segment `seg` of a sequence of n: chunks [c0, c1).
__device__ __forceinline__ void decay_span(int n, int seg, int seg_chunks, int* c0, int* c1) {
    const int all = (n + kDecayChunk - 1) / kDecayChunk;
    *c0 = min(seg * seg_chunks, all);
    *c1 = min(*c0 + seg_chunks, all);
}

// The chunked form.  One CTA per (pass, head, 64 value features, segment) walks
// its chunks of 128 tokens with the state in registers.  With L the decay and,
// for a chunk of n tokens in their order of walking, pos = 0 .. n - 1:
//   A    = X Y^T                              tensor memory
//   P_ij = scale A_ij L^(pos_i - pos_j)       pos_j <= pos_i, 16-bit
//   OX   = X S                                S: 16-bit copy of the state
//   O_i  = L^(pos_i + 1) OX_i + (P Z)_i
//   S   <- L^n S + Y^T Zh,   Zh_j = L^(n - 1 - pos_j) Z_j
// Backwards (a gradient G for S) the token's own term enters before the decay:
// OX_i is weighted with L^pos_i and Zh_j with scale L^(n - pos_j).
//
// The state is an fp32 result of its own, so Zh must not be rounded to the
// 16-bit type (one bf16 piece of it would be off by up to 2^-8, two by 2^-16): it
// goes to the tensor cores as two (fp16, 22 bits) or three (bf16, 24 bits) 16-bit
// pieces, side by side in the N extent of one product with Y, and the pieces' sums
// are added in fp32.  P, the copy of S that X meets and the result are rounded to the
// 16-bit type, half a step each: they only reach the 16-bit result.
//
// fp16 has no range for that by itself (terms of 1e-5 would be off by 1e-5 of themselves,
// weights of 1e-5 by 4e-3, a state or a weight past 65504 be lost).  What goes to the tensor
// cores is brought to the top of its range by exact powers of two:
//   Zh  for each chunk and 8 features, by their largest finite element; it leaves with the
//       sums in fp32, as the scale of a backward pass does.  A term keeps its 22 bits down
//       to 2^-17 of the largest, and is off by 2^-39 of that below
//   P   for each 16 rows, by the bound D max|X| max|Y| of their A, whose products the tensor
//       cores add in fp32, 2^-24 of it apart: a weight keeps its 11 bits down to 2^-28 of
//       the bound, and is off by 2^-39 of that below
//   S   for each chunk, by a bound that starts with the largest element and grows by 128
//       max|Y| max|Z| a chunk, as the state's own rounding errors do; likewise
// The maxima of X and Y are surveyed by the Zh warps, before Z lands.  (Exact maxima of P,
// over which the four warps of the same rows meet: 12 heads of 23400 tokens 84 us; the survey
// by a warp of its own 82, by the state warps 94; as it is 71; without P's and S's powers 65.)
//
// What bounds it: the chain of the roles from one chunk to the next, 4700 cycles of it at
// D = 128 (2.4 us a chunk), in which a role waits for what another hands over.  The
// products take about 2150 cycles of the tensor pipe; the operands they read, the loads,
// Zh, the state's copy and the staged result about 3100 cycles of shared-memory bandwidth.
// HBM would allow 1.3 us.
// Measured (one B200, device time of a replayed graph): 4 x 16 heads of 4096 tokens, d =
// 128, bf16: 86 us (269 MB and states: 3.1 TB/s), the gradients 235 us; 12 heads of 23400
// tokens, d = 64, fp16, in 12 segments: 71 us.  The first without Zh, P and stores: 57 us.
//
// Roles (eight warpgroups, 1024 threads): warp 0 loads (TMA), warp 1 issues the
// products, warp 2 stores (TMA), 3 fills rows past the end; 16 warps make P and the
// output (thread = token; each 32 keys of P and 16 features); 4 hold the state (thread =
// feature of y); 8 make Zh (bf16: thread = token, 32 features each; fp16: 8 features of
// all tokens, whose largest a warp then knows by itself; without P's and S's powers 12 heads
// of 23400 tokens take 64.8 us so, 67.5 with bf16's way and a barrier between the warps, 61.6
// without any).  Every role's work lies on the chain (Zh is written when its last reader is done),
// so it is spread over as many warps as the registers carry (8 row warps and 16 for Zh
// instead: 87.6 against 85.6 us for the large-head prompt).  Registers are dealt out
// between the warpgroups (setmaxnreg).
// Issue order: A_0, then per chunk Y^T Zh, X S, A of the next chunk, P Z: while the
// row warps read X S and hand over P, the next A runs, and the next P is made during
// P Z and Y^T Zh.  Every product has a completion barrier for either stage, on which
// all that depends on it waits, the reload of its operand included: X, Y and Z are
// each reloaded as soon as their last product is done.
//
// STATE: only the segment's own contribution to the state (from zero).
template <int D, bool BF16>
struct DecayCfg {
    static constexpr int NP = BF16 ? 3 : 2;             // pieces of Zh
    static constexpr uint32_t XB = D * 256u;            // X of a chunk
    static constexpr uint32_t YB = 32768u;              // Y; at D = 64 its upper half stays zero
    static constexpr uint32_t ZB = 16384u;              // 64 features of Z
    static constexpr uint32_t STAGE = XB + YB + ZB;
    static constexpr uint32_t OFF_ZH = 2 * STAGE;
    static constexpr uint32_t OFF_S = OFF_ZH + NP * ZB;  // D rows of 64 features
    // The result is staged for its TMA store in a buffer of its own or, where shared
    // memory is full (bf16, D = 128), in its step's Z, whose reload then waits for
    // the store (at D = 64 a buffer of its own takes a long prompt from 83 to 70 us;
    // at D = 128 half of X's stage instead of Z's: forward 85.3 to 84.6, gradients
    // 232 to 245 us).
    static constexpr bool OWN_O = D == 64 || !BF16;
    static constexpr uint32_t OFF_O = OWN_O ? OFF_S + D * 128u : XB + YB;
    static constexpr uint32_t O_STEP = OWN_O ? 0u : STAGE;
    static constexpr uint32_t OFF_PW = OFF_S + D * 128u + (OWN_O ? 16384u : 0u); // 32 zeros, L^0 .. L^128, L^31 .. L^0
    static constexpr uint32_t OFF_BAR = OFF_PW + (32 + 132 + 32) * 4;
    // two each of the loads and the products (by step parity), one of the rest
    static constexpr int B_XF = 0, B_YF = 2, B_ZF = 4, B_AF = 6, B_KVF = 8, B_QSD = 10, B_OD = 12,
                         B_PF = 14, B_ZH = 15, B_KVE = 16, B_SSF = 17, B_OE = 18, B_DR = 19, B_OR = 20,
                         B_OW = 22, B_SV = 24, B_SM = 26, NBAR = BF16 ? 24 : 27;
    // fp16: what takes Z's power of two out of the sums of each 8 features, of four chunks
    // (the state warps may still read a chunk's when the Zh warps are two on)
    static constexpr uint32_t OFF_ZD = (OFF_BAR + NBAR * 8 + 15) / 16 * 16;
    // the largest |X| of each 16 tokens and the largest |Y|, of four steps; what takes the
    // state copy's power out, of two; the largest |S| that each state warp begins with
    static constexpr uint32_t OFF_SX = OFF_ZD + 4 * 8 * 4, OFF_SY = OFF_SX + 4 * 8 * 4, OFF_SM = OFF_SY + 4 * 4,
                              OFF_SD = OFF_SM + 4 * 4;
    static constexpr uint32_t OFF_MISC = BF16 ? OFF_ZD : OFF_SD + 2 * 4;
    static constexpr uint32_t SMEM_BYTES = OFF_MISC + 16 + 1024;
    static constexpr uint32_t COL_KV = 256, COL_O = 448;  // tensor memory: A at 0 and 128
    static constexpr int NROW = 512, NSTATE = 128, NZH = 256, NTHREADS = 1024;
    // registers of a thread by role; the launch gives each of the eight warpgroups 64
    static constexpr int R_ISSUE = BF16 ? 32 : 40, R_ROW = 56, R_STATE = BF16 ? 144 : 136, R_ZH = 56;
    static_assert(R_ISSUE + 4 * R_ROW + R_STATE + 2 * R_ZH <= 8 * 64, "more registers than the launch has");
    static_assert(R_ISSUE <= 64 && R_ROW <= 64 && R_ZH <= 64 && R_STATE >= 64, "a share on the launch's wrong side");
    static_assert(SMEM_BYTES <= 232448u, "dynamic shared memory above the sm_100 per-block limit");
};

template <int D, bool BF16, bool STATE>
__global__ void __launch_bounds__(1024, 1)
    decay_chunk_kernel(const __grid_constant__ DecayMaps maps, const __grid_constant__ DecayParams p) {
    using C = DecayCfg<D, BF16>;
    constexpr int HALVES = D / 64, NP = C::NP;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // halves of a head next to each other, then the passes of a head: what they
    // share is read while it is in L2
    int id = blockIdx.x;
    const int hf = id % HALVES;
    id /= HALVES;
    const int pi = id % p.passes;
    id /= p.passes;
    const int bh = id % (p.B * p.H), seg = id / (p.B * p.H);
    const DecayPass& ps = p.pass[pi];
    const bool rev = ps.reverse != 0;
    const int len = decay_len(p.lens, bh / p.H, p.N);
    int c0, c1;
    decay_span(len, seg, p.seg_chunks, &c0, &c1);
    const int nch = c1 - c0;
    // chunk of step i, and its number of tokens
    auto chunk = [&](int i) { return rev ? c1 - 1 - i : c0 + i; };
    auto tokens = [&](int i) { return min(kDecayChunk, len - chunk(i) * kDecayChunk); };
    const uint32_t bar0 = base + C::OFF_BAR;
#define DBAR(i) (bar0 + 8u * static_cast<uint32_t>(i))
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + C::OFF_MISC);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    float* pw = reinterpret_cast<float*>(gbase + C::OFF_PW) + 32;
    const double ld = decay_log(p.log_decay, bh % p.H);
    float* zd = reinterpret_cast<float*>(gbase + C::OFF_ZD);
    float* sd = reinterpret_cast<float*>(gbase + C::OFF_SD);
    float* sx = reinterpret_cast<float*>(gbase + C::OFF_SX);
    float* sy = reinterpret_cast<float*>(gbase + C::OFF_SY);
    // of step i: Y (what 0), X (1), Z (2)
    auto load = [&](int i, int what) {
        const int s = i & 1, row = chunk(i) * kDecayChunk;
        const uint32_t sx = base + s * C::STAGE, sy = sx + C::XB, sz = sy + C::YB;
        if (what == 2) {
            mbar_arrive_expect_tx(DBAR(C::B_ZF + s), C::ZB);
            tma_load_3d(sz, &maps.m[ps.z], DBAR(C::B_ZF + s), hf * 64, row, bh);
        } else if (what == 0 || !STATE) {
            const uint32_t bar = DBAR((what ? C::B_XF : C::B_YF) + s);
            mbar_arrive_expect_tx(bar, D * 256u);
#pragma unroll
            for (int kb = 0; kb < HALVES; ++kb)
                tma_load_3d((what ? sx : sy) + kb * 16384u, &maps.m[what ? ps.x : ps.y], bar, kb * 64, row, bh);
        }
    };
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NBAR; ++i) {
            const int rows = i == C::B_PF || i == C::B_OE || i == C::B_OW || i == C::B_OW + 1;
            const int state = i == C::B_KVE || i == C::B_SSF;
            mbar_init(DBAR(i), rows ? C::NROW
                                    : (state ? C::NSTATE
                                             : (i == C::B_ZH ? C::NZH : (i == C::B_SM ? 4 : (i >= C::B_SV ? 8 : 1)))));
        }
        *abort_flag = 0u;
        if (!BF16)
            for (int i = 0; i < 4; ++i) sy[i] = 0.f;
        fence_mbar_init();
        // both stages are empty: their loads run while the tables are made
        for (int i = 0; i < 2 && i < nch; ++i)
            for (int what = 0; what < 3; ++what) load(i, what);
    }
    // L^m; the product's rounding error enters as a correction, so a power's error
    // stays that of the exponential
    for (int m = threadIdx.x; m <= kDecayChunk; m += C::NTHREADS) {
        const float l1 = static_cast<float>(ld), x = l1 * m;
        pw[m] = expf(x) * (1.f + fmaf(l1, static_cast<float>(m), -x));
        if (m < 32) pw[132 + 31 - m] = pw[m], pw[-1 - m] = 0.f;
    }
    if (D == 64) {  // features 64-127 of Y: zeros that no load touches
        for (int i = threadIdx.x; i < 2 * 1024; i += C::NTHREADS)
            *reinterpret_cast<uint4*>(gbase + (i >> 10) * C::STAGE + C::XB + 16384u + (i & 1023) * 16) =
                make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_smem();
    }
    if (warp == 1) {
        tmem_alloc(base + C::OFF_MISC, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if constexpr (STATE) cudaTriggerProgrammaticLaunchCompletion();
    if (warp < 4) regs_down<C::R_ISSUE>();
    if (warp == 0) {
        // ------------------------------------------------------ TMA producer
        if (elect_one()) {
            bool ok = true;
            int issued = 3 * min(nch, 2);
            for (int i = 2; i < nch; ++i) {
                const int s = i & 1;
                const uint32_t par = ((i >> 1) - 1) & 1;
                if (!(ok = wait_bounded(DBAR(C::B_KVF + s), par, abort_flag))) break;
                load(i, 0);
                issued = 3 * i + 1;
                if (!STATE && !(ok = wait_bounded(DBAR(C::B_QSD + s), par, abort_flag))) break;
                load(i, 1);
                issued = 3 * i + 2;
                if (!STATE && !(ok = wait_bounded(DBAR((C::OWN_O ? C::B_OD : C::B_OR) + s), par, abort_flag))) break;
                load(i, 2);
                issued = 3 * i + 3;
            }
            if (!ok) {  // let the copies in flight land before the CTA exits
                for (int k = issued > 6 ? issued - 6 : 0; k < issued; ++k) {
                    const int i = k / 3, what = k % 3;
                    if (STATE && what == 1) continue;
                    const int b = what == 0 ? C::B_YF : (what == 1 ? C::B_XF : C::B_ZF);
                    wait_drain(DBAR(b + (i & 1)), (i >> 1) & 1);
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------- MMA issuer
        if (elect_one()) {
            constexpr uint32_t ID_A = idesc_f16(BF16, 128, 128, false, false);     // X Y^T
            constexpr uint32_t ID_KV = idesc_f16(BF16, 128, 64 * NP, true, true);  // Y^T Zh
            constexpr uint32_t ID_O = idesc_f16(BF16, 128, 64, false, true);       // X S, P Z
            // descriptors of X and, transposed, of Y and Z of either stage, of Zh and of
            // the state's copy; a step along them is an addition to the address
            // (no arrays of them: indexed by the stage they would live in local memory)
            const uint64_t dx = sdesc_sw128(base, 16, 1024), dy = sdesc_sw128(base + C::XB, 16384, 1024);
            constexpr uint32_t ST16 = C::STAGE >> 4;
            const uint64_t dzh = sdesc_sw128(base + C::OFF_ZH, 16384, 1024);
            const uint64_t dst = sdesc_sw128(base + C::OFF_S, 16384, 1024);
            // A of step i into its buffer, last read by the P Z of step i - 2; in
            // a chunk that is not full, the rows past its end are cleared first
            auto issue_a = [&](int i) -> bool {
                const int s = i & 1;
                if (!wait3(DBAR(C::B_XF + s), (i >> 1) & 1, true, DBAR(C::B_YF + s), (i >> 1) & 1, true,
                           DBAR(C::B_OD + s), ((i >> 1) - 1) & 1, i >= 2, abort_flag))
                    return false;
                if (!BF16 && !wait_bounded(DBAR(C::B_SV + s), (i >> 1) & 1, abort_flag)) return false;
                if (tokens(i) < kDecayChunk && !wait_bounded(DBAR(C::B_ZH), i & 1, abort_flag)) return false;
                tc_fence_after();
                const uint64_t x = dx + s * ST16, y = x + (C::XB >> 4);
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * 16384u + (kk & 3) * 32u) >> 4;
                    mma_ss(tmem + 128u * s, x + off, y + off, ID_A, kk > 0 ? 1u : 0u);
                }
                mma_commit(DBAR(C::B_AF + s));
                return true;
            };
            bool ok = true;
            if constexpr (!STATE) ok = nch == 0 || issue_a(0);
            for (int i = 0; ok && i < nch; ++i) {
                const int s = i & 1;
                // Zh written, the previous sums read by the state warps
                if (!(ok = wait3(DBAR(C::B_ZH), i & 1, true, DBAR(C::B_KVE), (i - 1) & 1, i >= 1,
                                 DBAR(C::B_YF + s), (i >> 1) & 1, STATE, abort_flag)))
                    break;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < 8; ++kk)  // 16 tokens (2048 bytes) per step
                    mma_ss(tmem + C::COL_KV, dy + s * ST16 + kk * 128u, dzh + kk * 128u, ID_KV, kk > 0 ? 1u : 0u);
                mma_commit(DBAR(C::B_KVF + s));
                if constexpr (!STATE) {
                    // the state's copy stored, the previous output read
                    if (!(ok = wait3(DBAR(C::B_SSF), i & 1, true, DBAR(C::B_OE), (i - 1) & 1, i >= 1, 0u, 0u,
                                     false, abort_flag)))
                        break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = ((kk >> 2) * 16384u + (kk & 3) * 32u) >> 4;
                        mma_ss(tmem + C::COL_O, dx + s * ST16 + off, dst + kk * 128u, ID_O, kk > 0 ? 1u : 0u);
                    }
                    mma_commit(DBAR(C::B_QSD + s));
                    if (i + 1 < nch && !(ok = issue_a(i + 1))) break;
                    // P written and X S read: P Z takes its columns
                    if (!(ok = wait_bounded(DBAR(C::B_PF), i & 1, abort_flag))) break;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)
                        mma_ts(tmem + C::COL_O, tmem + 128u * s + (kk >> 1) * 32u + (kk & 1) * 8u,
                               dy + s * ST16 + (C::YB >> 4) + kk * 128u, ID_O, kk > 0 ? 1u : 0u);
                    mma_commit(DBAR(C::B_OD + s));
                }
            }
            if (!ok) {  // every issued MMA must finish before tensor memory is freed
                mma_commit(DBAR(C::B_DR));
                wait_drain(DBAR(C::B_DR), 0);
            }
        }
        __syncwarp();
    } else if (warp == 2) {
        // ---------------------------------------------------------- output
        // O_i leaves its staging by TMA
        if (!STATE && elect_one()) {
            for (int i = 0; i < nch; ++i) {
                const int s = i & 1;
                if (!wait_bounded(DBAR(C::B_OW + s), (i >> 1) & 1, abort_flag)) break;
                if (tokens(i) == kDecayChunk) {
                    tma_store_3d(&maps.m[ps.out_map], base + C::OFF_O + s * C::O_STEP, hf * 64,
                                 chunk(i) * kDecayChunk, bh);
                    bulk_commit();
                    bulk_wait_read_all();
                }
                mbar_arrive(DBAR(C::B_OR + s));
            }
            bulk_wait_all();
        }
        __syncwarp();
    } else if (warp < 4) {
        // the rows of this segment past the sequence's end, if they are to be zeros (a
        // fill of its own in front of the call: 54 us instead of 43 for the gradients of
        // 8 x 12 heads to 1024 tokens)
        if (!STATE && p.zero_past) {
            const int whole = p.seg_chunks * kDecayChunk;
            const int end = min(p.N - seg * whole, whole);
            uint8_t* out = static_cast<uint8_t*>(ps.out) +
                           (static_cast<size_t>(bh) * p.N + seg * whole) * (D * 2) + hf * 128 + (lane & 7) * 16;
            for (int r = max(len - seg * whole, 0) + (lane >> 3); r < end; r += 4)
                *reinterpret_cast<uint4*>(out + static_cast<size_t>(r) * (D * 2)) = make_uint4(0u, 0u, 0u, 0u);
        }
    } else if (warp < 20) {
        // ----------------------------------------- P and the output (rows)
        regs_down<C::R_ROW>();
        const int cb = (warp - 4) >> 2;        // keys 32 cb.. of P, features 16 cb.. of O
        const int wq = warp & 3, r = wq * 32 + lane;
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(wq * 32) << 16);
        const float* near = rev ? pw : pw + 132;
        // L^-31 out of range (fp16: with P's power of two times scale, 2^63 at most, since no
        // fp16 number but 0 is below 2^-24)
        const bool steep = pw[31] < (BF16 ? 0x1p-100f : 0x1p-60f);
        uint32_t o16[8] = {};  // the output of a step, until it is staged
        auto stage = [&](int i) -> bool {
            const int b = i & 1, n = tokens(i);
            // the staging's previous content has left
            if (C::OWN_O && i >= 1 &&
                !__all_sync(0xffffffffu, wait_bounded(DBAR(C::B_OR + (b ^ 1)), ((i - 1) >> 1) & 1, abort_flag)))
                return false;
            if (n == kDecayChunk) {
                // as the TMA store expects it: 16-byte piece j of row r at j ^ (r mod 8).
                // Stored from registers, 32 bytes of each row by a thread, every store was
                // 32 wavefronts of L1: 31 of the large-head prompt's 103 us.
                uint8_t* dst = gbase + C::OFF_O + b * C::O_STEP + r * 128;
                *reinterpret_cast<uint4*>(dst + (((2 * cb) ^ (r & 7)) << 4)) = make_uint4(o16[0], o16[1], o16[2], o16[3]);
                *reinterpret_cast<uint4*>(dst + (((2 * cb + 1) ^ (r & 7)) << 4)) =
                    make_uint4(o16[4], o16[5], o16[6], o16[7]);
                fence_proxy_async_smem();
            } else if (r < n) {  // rows past the sequence's end stay as they are
                uint4* dst = reinterpret_cast<uint4*>(
                    static_cast<uint8_t*>(ps.out) +
                    (static_cast<size_t>(bh) * p.N + chunk(i) * kDecayChunk + r) * (D * 2) + hf * 128 + cb * 32);
                dst[0] = make_uint4(o16[0], o16[1], o16[2], o16[3]);
                dst[1] = make_uint4(o16[4], o16[5], o16[6], o16[7]);
            }
            mbar_arrive(DBAR(C::B_OW + b));
            return true;
        };
        bool ok = true;
        for (int i = 0; !STATE && i < nch; ++i) {
            const int b = i & 1, n = tokens(i);
            if (!(ok = __all_sync(0xffffffffu, wait_bounded(DBAR(C::B_AF + b), (i >> 1) & 1, abort_flag)))) break;
            float pscale = p.scale, pup = 1.f;
            if constexpr (!BF16) {
                // what bounds the row's A
                pup = fp16_up(sx[(i & 3) * 8 + (r >> 4)] * sy[i & 3] * (D * p.scale));
                pscale *= pup;
            }
            tc_fence_after();
            {
                const uint32_t col = lane_addr + 128u * b + 32u * cb;
                uint32_t pk[16];
                if (rev ? cb < wq : cb > wq) {  // 32 keys behind all rows of the warp
#pragma unroll
                    for (int e = 0; e < 16; ++e) pk[e] = 0u;
                } else {
                    uint32_t v[32];
                    tmem_ld32(col, v);
                    tmem_ld_wait();
                    reg_fence32(v);
                    if (cb == wq && steep) {
#pragma unroll
                        for (int e = 0; e < 32; ++e) {
                            const int gap = rev ? e - lane : lane - e;  // zeros in front of L^0
                            const float x = __uint_as_float(v[e]) * (pw[gap] * pscale);
                            v[e] = gap >= 0 ? __float_as_uint(x) : 0u;
                        }
                    } else {
                        // L^(distance) as L^(from the row to the block's near end) times
                        // L^(from there to the key): neither above 1 behind the row, and in
                        // the row's own block the first at most L^-31
                        const float u = cb == wq ? pscale / pw[rev ? lane : 31 - lane]
                                                 : pscale * (rev ? pw[cb * 32 - r] : pw[r - cb * 32 - 31]);
                        const uint64_t u2 = f2(u, u);
#pragma unroll
                        for (int e = 0; e < 32; e += 4) {
                            const float4 w = *reinterpret_cast<const float4*>(near + e);
                            const float2 a = unf2(mul2(f2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])),
                                                       mul2(u2, f2(w.x, w.y))));
                            const float2 c = unf2(mul2(f2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])),
                                                       mul2(u2, f2(w.z, w.w))));
                            v[e] = __float_as_uint(a.x), v[e + 1] = __float_as_uint(a.y);
                            v[e + 2] = __float_as_uint(c.x), v[e + 3] = __float_as_uint(c.y);
                        }
                        if (cb == wq) {
                            const uint32_t seen = rev ? 0xffffffffu << lane : 0xffffffffu >> (31 - lane);
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(seen & (1u << e))) v[e] = 0u;
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        pk[e] = pack2<BF16>(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
                }
                tmem_st16(col, pk);  // over columns already read
                tmem_st_wait();
            }
            // X S, before P Z takes its columns
            if (!(ok = __all_sync(0xffffffffu, wait_bounded(DBAR(C::B_QSD + b), (i >> 1) & 1, abort_flag)))) break;
            tc_fence_after();
            uint32_t ox[16], v[16];
            tmem_ld16(lane_addr + C::COL_O + 16u * cb, ox);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) reg_fence(ox[e]);
            float w = r < n ? (rev ? pw[n - 1 - r] : pw[r + 1]) : 0.f, down = 1.f;
            if (!BF16) w *= sd[b], down = fp16_down(pup);
            tc_fence_before();
            mbar_arrive(DBAR(C::B_PF));
            // in a buffer of its own the previous step's output is staged during P Z
            // (12 heads of 23400 tokens, before the powers of two: 64.2 to 62.9 us)
            if (C::OWN_O && i >= 1 && !(ok = stage(i - 1))) break;
            if (!(ok = __all_sync(0xffffffffu, wait_bounded(DBAR(C::B_OD + b), (i >> 1) & 1, abort_flag)))) break;
            tc_fence_after();
            tmem_ld16(lane_addr + C::COL_O + 16u * cb, v);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) reg_fence(v[e]);
            tc_fence_before();
            mbar_arrive(DBAR(C::B_OE));
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if constexpr (BF16) {
                    o16[e] = pack2<BF16>(fmaf(w, __uint_as_float(ox[2 * e]), __uint_as_float(v[2 * e])),
                                         fmaf(w, __uint_as_float(ox[2 * e + 1]), __uint_as_float(v[2 * e + 1])));
                } else {
                    const float2 f = unf2(fma2(
                        f2(w, w), f2(__uint_as_float(ox[2 * e]), __uint_as_float(ox[2 * e + 1])),
                        mul2(f2(down, down), f2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1])))));
                    o16[e] = pack2<BF16>(f.x, f.y);
                }
            }
            if (!C::OWN_O && !(ok = stage(i))) break;
        }
        if (C::OWN_O && !STATE && ok && nch > 0) stage(nch - 1);
    } else if (warp < 24) {
        // -------------------------------------------------------- the state
        regs_up<C::R_STATE>();
        const int a = (warp & 3) * 32 + lane;  // feature of y == TMEM lane
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const size_t mat = static_cast<size_t>(bh) * D * D;
        const size_t seg_mat = (static_cast<size_t>(pi) * p.nseg + seg) * p.B * p.H * D * D + mat;
        float copy = rev ? 1.f : p.scale;
        float bound = 0.f;  // fp16: of |S|
        bool ok = true;
        uint64_t st[32];  // features 2 c, 2 c + 1 of z
#pragma unroll
        for (int c = 0; c < 32; ++c) st[c] = 0ull;
        if (!STATE && a < D) {
            if (p.nseg == 1 && ps.init && ps.transposed) {
#pragma unroll
                for (int c = 0; c < 32; ++c)
                    st[c] = f2(ps.init[mat + (hf * 64 + 2 * c) * D + a], ps.init[mat + (hf * 64 + 2 * c + 1) * D + a]);
            } else if (p.nseg > 1 || ps.init) {
                if (p.nseg > 1) cudaGridDependencySynchronize();  // the scan's result, all else is the call's input
                const float4* src = reinterpret_cast<const float4*>((p.nseg > 1 ? p.seg + seg_mat : ps.init + mat) +
                                                                    a * D + hf * 64);
#pragma unroll
                for (int c = 0; c < 16; ++c) {
                    const float4 f = src[c];
                    st[2 * c] = f2(f.x, f.y), st[2 * c + 1] = f2(f.z, f.w);
                }
            }
        }
        // row a of the state's 16-bit copy: eight 16-byte pieces placed by the
        // 128-byte swizzle (piece j at j ^ (a mod 8))
        auto store_copy = [&](int i) {
            if constexpr (!BF16) {  // by a power of two, which leaves with the scale
                copy = fp16_up(bound);
                if (warp == 20 && lane == 0) sd[i & 1] = (rev ? 1.f : p.scale) * fp16_down(copy);
            }
            if (a < D) {
                uint8_t* srow = gbase + C::OFF_S + a * 128;
                const uint64_t c2 = f2(copy, copy);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = unf2(mul2(st[4 * j + e], c2));
                        w[e] = pack2<BF16>(f.x, f.y);
                    }
                    *reinterpret_cast<uint4*>(srow + ((j ^ (a & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(DBAR(C::B_SSF));
        };
        if (!BF16 && !STATE && (p.nseg > 1 || ps.init)) {
            // the largest |S| to begin with: the warps meet once
            float top = 0.f;  // (a maximum passes over NaN)
#pragma unroll
            for (int c = 0; c < 32; ++c) {
                const float2 f = unf2(st[c]);
                top = max3(top, fabsf(f.x), fabsf(f.y));
            }
            const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
            float4* sm = reinterpret_cast<float4*>(gbase + C::OFF_SM);
            if (lane == 0) {
                (&sm->x)[warp & 3] = __uint_as_float(bits);
                mbar_arrive(DBAR(C::B_SM));
            }
            ok = __all_sync(0xffffffffu, wait_bounded(DBAR(C::B_SM), 0, abort_flag));
            const float4 m = *sm;
            bound = fmaxf(max3(m.x, m.y, m.z), m.w);
            if (isinf(bound)) bound = 16384.f;  // an infinity: the state as it is
        }
        if constexpr (!STATE) store_copy(0);
        const double full = exp(ld * kDecayChunk);
        for (int i = 0; ok && i < nch; ++i) {
            // the sums of step i into the state: S <- L^n S + sums, L^n as a pair of
            // floats so that its error does not add up over the chunks
            if (!(ok = __all_sync(0xffffffffu, wait_bounded(DBAR(C::B_KVF + (i & 1)), (i >> 1) & 1, abort_flag))))
                break;
            tc_fence_after();
            const double gd = tokens(i) == kDecayChunk ? full : exp(ld * tokens(i));
            const float gf = static_cast<float>(gd);
            const uint64_t g = f2(gf, gf), g2 = f2(static_cast<float>(gd - gf), static_cast<float>(gd - gf));
            float largest = 0.f;  // times 2^15 a bound of |Z| times its scale
#pragma unroll
            for (int cc = 0; cc < 4; ++cc) {
                uint32_t v[NP][16];
#pragma unroll
                for (int k = 0; k < NP; ++k) tmem_ld16(lane_addr + C::COL_KV + 64u * k + 16u * cc, v[k]);
                const float2 down = BF16 ? make_float2(1.f, 1.f)
                                         : *reinterpret_cast<const float2*>(zd + (i & 3) * 8 + 2 * cc);
                if (!BF16) largest = max3(largest, down.x, down.y);
                tmem_ld_wait();
#pragma unroll
                for (int k = 0; k < NP; ++k)
#pragma unroll
                    for (int e = 0; e < 16; ++e) reg_fence(v[k][e]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    uint64_t sum = f2(__uint_as_float(v[NP - 1][2 * e]), __uint_as_float(v[NP - 1][2 * e + 1]));
#pragma unroll
                    for (int k = NP - 2; k >= 0; --k)  // the small pieces first
                        sum = add2(sum, f2(__uint_as_float(v[k][2 * e]), __uint_as_float(v[k][2 * e + 1])));
                    if (!BF16) sum = mul2(sum, e < 4 ? f2(down.x, down.x) : f2(down.y, down.y));
                    uint64_t& x = st[8 * cc + e];
                    x = fma2(g, x, fma2(g2, x, sum));
                }
            }
            if constexpr (!BF16 && !STATE) {
                // an entry of the sums: 128 terms of |Y| and |Zh| at most
                bound = fmaf(gf, bound, 0x1p22f * largest * sy[i & 3]);
            }
            tc_fence_before();
            mbar_arrive(DBAR(C::B_KVE));
            if (!STATE && i + 1 < nch) {
                // the copy was last read by X S of this step
                if (!(ok = __all_sync(0xffffffffu, wait_bounded(DBAR(C::B_QSD + (i & 1)), (i >> 1) & 1, abort_flag))))
                    break;
                store_copy(i + 1);
            }
        }
        float* last = STATE ? p.seg + seg_mat : (p.nseg == 1 && ps.last ? ps.last + mat : nullptr);
        if (ok && last && a < D) {
            float4* dst = reinterpret_cast<float4*>(last + a * D + hf * 64);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
                const float2 f = unf2(st[2 * c]), h = unf2(st[2 * c + 1]);
                dst[c] = make_float4(f.x, f.y, h.x, h.y);
            }
        }
    } else {
        // -------------------------------------------------------------- Zh
        regs_down<C::R_ZH>();
        // four 16-byte pieces (8 features of a token) a thread: bf16, four of one token;
        // fp16, the same features of four tokens, so that a warp by itself knows the
        // largest element of its 8 features
        auto token = [&](int t) { return BF16 ? (warp & 3) * 32 + lane : 32 * t + lane; };
        auto piece = [&](int t) { return BF16 ? ((warp - 24) >> 2 << 2) + t : warp - 24; };
        auto at = [&](int t) { return static_cast<uint32_t>(token(t) * 128 + ((piece(t) ^ (token(t) & 7)) << 4)); };
        for (int i = 0; i < nch; ++i) {
            const int s = i & 1, n = tokens(i);
            uint8_t* zt = gbase + s * C::STAGE + C::XB + C::YB;
            uint8_t* ht = gbase + C::OFF_ZH;
            if constexpr (!BF16 && !STATE) {
                // survey, before Z lands: the largest |X| and |Y|, 16 tokens a warp (rows of 128
                // bytes, whatever their pieces' order: lane = row mod 4, piece)
                if (!__all_sync(0xffffffffu, wait_bounded(DBAR(C::B_XF + s), (i >> 1) & 1, abort_flag) &&
                                                 wait_bounded(DBAR(C::B_YF + s), (i >> 1) & 1, abort_flag)))
                    break;
                const int row = (warp - 24) * 16 + (lane >> 3);
                const uint8_t* src = gbase + s * C::STAGE + (warp - 24) * 2048 + lane * 16;
                __half2 m[2][2];  // (a maximum passes over NaN)
#pragma unroll
                for (int e = 0; e < 4; ++e) m[e >> 1][e & 1] = __float2half2_rn(0.f);
#pragma unroll
                for (int h = 0; h < HALVES; ++h) {
                    uint4 x[8];  // all loads before the first is used
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        x[u] = make_uint4(0u, 0u, 0u, 0u);
                        if (row + 4 * (u & 3) < n)
                            x[u] = *reinterpret_cast<const uint4*>(src + (u >> 2) * C::XB + h * 16384 + (u & 3) * 512);
                    }
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            m[u >> 2][e & 1] =
                                __hmax2(m[u >> 2][e & 1], __habs2(*reinterpret_cast<const __half2*>(&w[e])));
                    }
                }
                uint32_t top[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const __half2 a = __hmax2(m[k][0], m[k][1]);
                    top[k] = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(__half_as_ushort(
                                                                __hmax(__low2half(a), __high2half(a)))));
                }
                if (lane == 0) {  // (an infinity as fp16's largest)
                    sx[(i & 3) * 8 + warp - 24] = unpack2<false>(min(top[0], 0x7bffu)).x;
                    atomicMax(reinterpret_cast<uint32_t*>(sy + (i & 3)),
                              __float_as_uint(unpack2<false>(min(top[1], 0x7bffu)).x));
                }
                if (lane == 0) mbar_arrive(DBAR(C::B_SV + s));
            }
            // Z landed
            bool ok = wait_bounded(DBAR(C::B_ZF + s), (i >> 1) & 1, abort_flag);
            uint4 in[4];
            float up = rev ? p.scale : 1.f;
            auto load_z = [&]() {
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    in[t] = token(t) < n ? *reinterpret_cast<const uint4*>(zt + at(t)) : make_uint4(0u, 0u, 0u, 0u);
            };
            if constexpr (!BF16) {
                if (!__all_sync(0xffffffffu, ok)) break;
                load_z();
                __half2 top2 = __float2half2_rn(0.f);  // (its maximum passes over NaN)
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    const uint32_t z[4] = {in[t].x, in[t].y, in[t].z, in[t].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) top2 = __hmax2(top2, __habs2(*reinterpret_cast<const __half2*>(&z[e])));
                }
                const float2 tf = __half22float2(top2);
                uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(fmaxf(tf.x, tf.y)));
                if (top >= 0x7f800000u) {  // an infinity: the largest finite one
                    float most = 0.f;
#pragma unroll
                    for (int t = 0; t < 4; ++t) {
                        const uint32_t z[4] = {in[t].x, in[t].y, in[t].z, in[t].w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = unpack2<false>(z[e]);
                            most = fmaxf(most, isfinite(f.x) ? fabsf(f.x) : 0.f);
                            most = fmaxf(most, isfinite(f.y) ? fabsf(f.y) : 0.f);
                        }
                    }
                    top = __reduce_max_sync(0xffffffffu, __float_as_uint(most));
                }
                const float down = up;
                up = fp16_up(__uint_as_float(top));
                if (lane == 0) zd[(i & 3) * 8 + piece(0)] = top > 0u ? down * fp16_down(up) : 0.f;
            }
            // the previous product has read Zh
            ok = ok && (i == 0 || wait_bounded(DBAR(C::B_KVF + (s ^ 1)), ((i - 1) >> 1) & 1, abort_flag));
            if (n < kDecayChunk)  // Y is cleared below
                ok = ok && wait_bounded(DBAR(C::B_YF + s), (i >> 1) & 1, abort_flag);
            if (!__all_sync(0xffffffffu, ok)) break;
            if constexpr (BF16) load_z();
            // the survey's slot of two steps on, last read for two steps back
            if (!BF16 && !STATE && warp == 24 && lane == 0) sy[(i + 2) & 3] = 0.f;
            const uint64_t minus = f2(-1.f, -1.f);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                // (past the end in is zero, whatever its weight)
                const float w = up * (rev ? pw[token(t) + 1] : pw[max(n - 1 - token(t), 0)]);
                const uint64_t w2 = f2(w, w);
                const uint32_t z[4] = {in[t].x, in[t].y, in[t].z, in[t].w};
                uint32_t out[NP][4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float2 zf = unpack2<BF16>(z[e]);
                    uint64_t f = mul2(f2(zf.x, zf.y), w2);
#pragma unroll
                    for (int k = 0; k < NP; ++k) {
                        const float2 x = unf2(f);
                        out[k][e] = pack2<BF16>(x.x, x.y);
                        const float2 h = unpack2<BF16>(out[k][e]);
                        f = fma2(f2(h.x, h.y), minus, f);
                    }
                }
#pragma unroll
                for (int k = 0; k < NP; ++k)
                    *reinterpret_cast<uint4*>(ht + k * C::ZB + at(t)) =
                        make_uint4(out[k][0], out[k][1], out[k][2], out[k][3]);
            }
            if (n < kDecayChunk) {
                // tokens past the end may hold anything, NaN included, in y and z
                const uint4 none = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if (token(t) < n) continue;
                    *reinterpret_cast<uint4*>(zt + at(t)) = none;
#pragma unroll
                    for (int k = 0; k < HALVES; ++k)
                        *reinterpret_cast<uint4*>(zt - C::YB + k * 16384u + at(t)) = none;
                }
            }
            fence_proxy_async_smem();
            mbar_arrive(DBAR(C::B_ZH));
        }
    }
#undef DBAR
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// The segments' own contributions (p.seg) into the state in front of each, in
// the order of walking, and into the state behind the last.  Thread = 4 entries;
// eight segments' loads are in flight before the first is used (one at a time: 24
// us for 12 segments of 12 heads).
template <int D>
__global__ void __launch_bounds__(128) decay_scan_kernel(const __grid_constant__ DecayParams p) {
    constexpr int PER = D * D / 4, AHEAD = 8;
    const int bh = blockIdx.y, pi = blockIdx.z;
    const int e4 = blockIdx.x * 128 + threadIdx.x;  // D * D / 4 is a multiple of 128
    const DecayPass& ps = p.pass[pi];
    const int len = decay_len(p.lens, bh / p.H, p.N);
    const double ld = decay_log(p.log_decay, bh % p.H);
    const size_t mat = static_cast<size_t>(bh) * PER;
    float4* at = reinterpret_cast<float4*>(p.seg) + static_cast<size_t>(pi) * p.nseg * p.B * p.H * PER + mat + e4;
    const size_t step = static_cast<size_t>(p.B) * p.H * PER;
    cudaTriggerProgrammaticLaunchCompletion();
    const int whole = p.seg_chunks * kDecayChunk;  // tokens of a full segment
    const double full = exp(ld * whole);
    float4 S = make_float4(0.f, 0.f, 0.f, 0.f);
    if (ps.init) {
        if (ps.transposed) {
            const int a = e4 * 4 / D, c = e4 * 4 % D;
            const float* src = ps.init + mat * 4 + a;
            S = make_float4(src[c * D], src[(c + 1) * D], src[(c + 2) * D], src[(c + 3) * D]);
        } else {
            S = reinterpret_cast<const float4*>(ps.init)[mat + e4];
        }
    }
    cudaGridDependencySynchronize();  // the segments' own contributions
    for (int i0 = 0; i0 < p.nseg; i0 += AHEAD) {
        float4 own[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int i = i0 + k, seg = ps.reverse ? p.nseg - 1 - i : i;
            if (i < p.nseg) own[k] = at[seg * step];
        }
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int i = i0 + k, seg = ps.reverse ? p.nseg - 1 - i : i;
            if (i >= p.nseg) break;
            int n = len - seg * whole;
            n = n < 0 ? 0 : (n > whole ? whole : n);
            const double gd = n == whole ? full : exp(ld * n);
            const float g = static_cast<float>(gd), g2 = static_cast<float>(gd - g);
            at[seg * step] = S;
            S.x = fmaf(g, S.x, fmaf(g2, S.x, own[k].x)), S.y = fmaf(g, S.y, fmaf(g2, S.y, own[k].y));
            S.z = fmaf(g, S.z, fmaf(g2, S.z, own[k].z)), S.w = fmaf(g, S.w, fmaf(g2, S.w, own[k].w));
        }
    }
    if (ps.last) reinterpret_cast<float4*>(ps.last)[mat + e4] = S;
}

// Segments of a call: one, unless its CTAs (one per pass, head and 64 features)
// fill less than half of the device's 148 multiprocessors; then as many as fit,
// of four chunks at least (a segment costs a second pass over y and z, and a
// state written and read: 12 heads of 23400 tokens, d = 64, take 71 us in 12
// segments; 183 chunks in a row are 370 us at the 2 us each that a long walk takes).
inline void decay_segments(int B, int H, int N, int d, int passes, int* nseg, int* seg_chunks) {
    const long long ctas = 1LL * passes * B * H * (d / 64);
    const int chunks = (N + kDecayChunk - 1) / kDecayChunk;
    long long n = ctas * 2 <= 148 ? 148 / ctas : 1;
    if (n > chunks / 4) n = chunks / 4;
    if (n < 1) n = 1;
    *seg_chunks = static_cast<int>((chunks + n - 1) / n);
    *nseg = (chunks + *seg_chunks - 1) / *seg_chunks;
}

inline size_t decay_workspace(int B, int H, int N, int d, int passes) {
    int nseg, seg_chunks;
    decay_segments(B, H, N, d, passes, &nseg, &seg_chunks);
    return nseg > 1 ? static_cast<size_t>(passes) * nseg * B * H * d * d * 4 : 0;
}

template <int D, bool BF16>
bool decay_set_attributes() {
    const int bytes = static_cast<int>(DecayCfg<D, BF16>::SMEM_BYTES);
    return cudaFuncSetAttribute(decay_chunk_kernel<D, BF16, false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                bytes) == cudaSuccess &&
           cudaFuncSetAttribute(decay_chunk_kernel<D, BF16, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                bytes) == cudaSuccess;
}

template <int D, bool BF16>
void decay_launch(const DecayMaps& maps, const DecayParams& p, cudaStream_t st) {
    constexpr uint32_t bytes = DecayCfg<D, BF16>::SMEM_BYTES;
    const unsigned grid = static_cast<unsigned>(p.B) * p.H * (D / 64) * p.passes * p.nseg;
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute early;  // a launch begins while the one before still runs (68 to 66 us)
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &early;
    cfg.stream = st;
    if (p.nseg > 1) {
        decay_chunk_kernel<D, BF16, true><<<grid, 1024, bytes, st>>>(maps, p);
        cfg.numAttrs = 1;
        cfg.gridDim = dim3(D * D / 512, p.B * p.H, p.passes);
        cfg.blockDim = dim3(128);
        cudaLaunchKernelEx(&cfg, decay_scan_kernel<D>, p);
    }
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(1024);
    cfg.dynamicSmemBytes = bytes;
    cudaLaunchKernelEx(&cfg, decay_chunk_kernel<D, BF16, false>, maps, p);
}

// One token: S <- g S + k v^T, o = scale q S, the state read and written once:
// bound by HBM (8 D^2 bytes a head; 128 x 16 heads of D = 128: 41 us, 6.5 TB/s).  One
// CTA per head and slice of 4 COLS4 columns (32: four CTAs a head at D = 128, so that a
// single sequence's 16 heads reach 64 multiprocessors: 2.1 us, where one CTA a head and
// a thread a column took 23); a thread holds 4 columns of D / ROWS rows, all loaded
// before the first is used; the ROWS partial sums of o meet in shared memory.
//
// g is a pair of floats, as a chunk's L^n is: the error of one, up to 2^-25, has the same
// sign at every token and adds up over the memory's length (2.6e-4 of a state after 20000
// tokens that forget 1e-4 each).  The pair is 1 + (g - 1) with g - 1 from expm1, whose own
// error adds up to a few 2^-24; below e^-1/2 a memory is too short for any to add up.  One
// thread makes it (16 heads of one sequence: 1.93 us a token, 1.84 with a single float; by
// exp in 64 bits 0.3 us more; by every thread the batch takes 42.8 us).
template <int D, bool BF16, int COLS4>
__global__ void __launch_bounds__(256) decay_step_kernel(const void* q, const void* k, const void* v,
                                                         const float* log_decay, const float* in,
                                                         float* out, void* o, int H, float scale) {
    constexpr int ROWS = 256 / COLS4, N = D / ROWS, SLICES = D / (4 * COLS4);
    __shared__ float sq[D], sk[D];
    __shared__ float4 so[ROWS][COLS4];
    __shared__ float2 sg;
    const int bh = blockIdx.x / SLICES, slice = blockIdx.x % SLICES;
    const int c = threadIdx.x % COLS4, r = threadIdx.x / COLS4, col = slice * 4 * COLS4 + 4 * c;
    const size_t at = static_cast<size_t>(bh) * D * D + static_cast<size_t>(r) * D + col;
    const float ld = decay_log(log_decay, bh % H);
    float4 s[N];
#pragma unroll
    for (int i = 0; i < N; ++i) s[i] = __ldcs(reinterpret_cast<const float4*>(in + at + i * ROWS * D));
    if (threadIdx.x < D / 2) {
        const size_t w = static_cast<size_t>(bh) * (D / 2) + threadIdx.x;
        const float2 a = unpack2<BF16>(static_cast<const uint32_t*>(q)[w]);
        const float2 b = unpack2<BF16>(static_cast<const uint32_t*>(k)[w]);
        sq[2 * threadIdx.x] = a.x, sq[2 * threadIdx.x + 1] = a.y;
        sk[2 * threadIdx.x] = b.x, sk[2 * threadIdx.x + 1] = b.y;
    }
    const uint2 zv = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(v) +
                                                     static_cast<size_t>(bh) * D + col);
    const float2 z0 = unpack2<BF16>(zv.x), z1 = unpack2<BF16>(zv.y);
    if (threadIdx.x == 255) {
        if (ld < -0.5f) {
            sg = make_float2(expf(ld), 0.f);
        } else {
            const float less = expm1f(ld), sum = 1.f + less;
            sg = make_float2(sum, less - (sum - 1.f));  // exact
        }
    }
    __syncthreads();
    const float g = sg.x, g2 = sg.y;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float a = sk[r + i * ROWS], b = sq[r + i * ROWS];
        s[i].x = fmaf(g, s[i].x, fmaf(g2, s[i].x, a * z0.x)), s[i].y = fmaf(g, s[i].y, fmaf(g2, s[i].y, a * z0.y));
        s[i].z = fmaf(g, s[i].z, fmaf(g2, s[i].z, a * z1.x)), s[i].w = fmaf(g, s[i].w, fmaf(g2, s[i].w, a * z1.y));
        __stcs(reinterpret_cast<float4*>(out + at + i * ROWS * D), s[i]);
        acc.x = fmaf(b, s[i].x, acc.x), acc.y = fmaf(b, s[i].y, acc.y);
        acc.z = fmaf(b, s[i].z, acc.z), acc.w = fmaf(b, s[i].w, acc.w);
    }
    so[r][c] = acc;
    __syncthreads();
    if (threadIdx.x < COLS4) {
        float4 sum = so[0][threadIdx.x];
#pragma unroll
        for (int i = 1; i < ROWS; ++i) {
            const float4 x = so[i][threadIdx.x];
            sum.x += x.x, sum.y += x.y, sum.z += x.z, sum.w += x.w;
        }
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(o) + static_cast<size_t>(bh) * D + col) =
            make_uint2(pack2<BF16>(sum.x * scale, sum.y * scale), pack2<BF16>(sum.z * scale, sum.w * scale));
    }
}

}  // namespace attn
