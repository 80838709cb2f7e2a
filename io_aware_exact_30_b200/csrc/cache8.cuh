// A paged key/value cache held in e4m3, one power-of-two scale for each page
// and head, and softmax attention over it.
//
// Layout: codes (num_pages, Hkv, page, D) bytes, scales (num_pages, Hkv) fp32,
// value = code * scale.  Slot s of a page holds one token; a sequence's token
// at position t lies in slot t % page of the page its table names at t / page.
//
// A power of two loses a floating code nothing but a binade at its subnormal
// end, and it is what makes a page that fills token by token sound: when a new
// token's largest value outgrows the page's scale, the held codes are moved to
// the new scale by an exact shift of their exponents (only codes that become
// subnormal round again), where an amax / 448 scale would round every held
// code a second time.
#pragma once

#include <cuda_fp8.h>

#include "ptx.cuh"

namespace attn {

constexpr int kErrPage = -11;  // ATTN_ERR_PAGE

// Records a bad page or length in the device error word unless it is taken.
__device__ __forceinline__ void record_bad_page() { atomicCAS(&g_attn_error, 0, kErrPage); }

// The least power of two s (not below 2^-126) with amax <= 448 s; 0 for 0.
// 448 = 1.75 * 2^8, so the exponent is that of amax less 8, plus one when the
// mantissa is above 1.75.
__device__ __forceinline__ float pow2_scale(float amax) {
    if (!(amax > 0.f)) return 0.f;
    const uint32_t bits = __float_as_uint(amax);
    int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    if (e < 1) e = 1;
    return __uint_as_float(static_cast<uint32_t>(e) << 23);
}

struct AppendParams {
    const uint8_t* x[2];   // new k, v: (B, Hkv, T, D) 16-bit
    uint8_t* codes[2];
    float* scale[2];
    const int* table;      // (B, max_pages)
    const int* lens;       // tokens held before, per sequence
    const int* n_new;      // tokens that come, per sequence; null: T
    int B, Hkv, T, num_pages, page, max_pages;
    int touched;           // pages that T tokens can touch: grid factor
};

// One CTA per (sequence, page its new tokens touch, head, K or V): no two CTAs
// share a page's codes or scale.  The page's new rows are read once, into
// registers (16 bytes a thread and step), while their largest magnitude is
// found; it decides the scale, and the rows are stored as codes.
//
// Bound by HBM for prompts (2 bytes read, 1 written per value: four of up to 4096
// tokens, 16 heads, d = 128: 26 us, 5.5 TB/s), for single tokens by the launch, two
// dependent loads and the parameters' copy in local memory, which the choice of K's or V's
// array at run time brings (64 sequences, 8 heads: 4.5 us).
template <int D, bool BF16, int NCH>
__global__ void __launch_bounds__(128) cache_append_kernel(const AppendParams p) {
    constexpr int PER_ROW = D / 8;  // 16-byte pieces of a row
    __shared__ uint32_t warp_max[4];
    long long id = blockIdx.x;
    const int w = static_cast<int>(id % p.touched);
    id /= p.touched;
    const int h = static_cast<int>(id % p.Hkv);
    id /= p.Hkv;
    const int kv = static_cast<int>(id & 1);
    const int b = static_cast<int>(id >> 1);
    const int len = p.lens[b];
    const int n = p.n_new ? p.n_new[b] : p.T;
    if (len < 0 || n < 0 || n > p.T) {
        if (w == 0 && h == 0 && kv == 0 && threadIdx.x == 0) record_bad_page();
        return;
    }
    const long long entry = len / p.page + static_cast<long long>(w);
    const long long p0 = entry * p.page;  // position of the page's slot 0
    const int s0 = len > p0 ? static_cast<int>(len - p0) : 0;
    const long long past = static_cast<long long>(len) + n - p0;
    const int s1 = past < p.page ? static_cast<int>(past) : p.page;
    if (s1 <= s0) return;
    const int id_page = entry < p.max_pages ? p.table[static_cast<size_t>(b) * p.max_pages + entry] : -1;
    if (id_page < 0 || id_page >= p.num_pages) {
        if (threadIdx.x == 0) record_bad_page();
        return;
    }
    const size_t slot = static_cast<size_t>(id_page) * p.Hkv + h;
    uint8_t* codes = p.codes[kv] + slot * p.page * D;
    float* scale = p.scale[kv] + slot;
    const uint8_t* rows = p.x[kv] + ((static_cast<long long>(b) * p.Hkv + h) * p.T + (p0 - len)) * D * 2;
    uint4 x[NCH];
    uint32_t top = 0u;  // the largest magnitude's bits, two 16-bit lanes
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = static_cast<int>(threadIdx.x) + 128 * i, s = c / PER_ROW;
        if (s >= s0 && s < s1) {
            x[i] = __ldg(reinterpret_cast<const uint4*>(rows) + c);
            top = __vmaxu2(top, x[i].x & 0x7fff7fffu);
            top = __vmaxu2(top, x[i].y & 0x7fff7fffu);
            top = __vmaxu2(top, x[i].z & 0x7fff7fffu);
            top = __vmaxu2(top, x[i].w & 0x7fff7fffu);
        }
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, m));
    if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = top;
    const float old = s0 > 0 ? *scale : 0.f;
    __syncthreads();
    top = __vmaxu2(__vmaxu2(warp_max[0], warp_max[1]), __vmaxu2(warp_max[2], warp_max[3]));
    constexpr uint32_t kFinite = BF16 ? 0x7f7f7f7fu : 0x7bff7bffu;  // the type's largest, twice
    if (__vmaxu2(top, kFinite) != kFinite) {
        // an element that is not finite becomes a NaN code; the scale is that of the others
        top = 0u;
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
            const int s = (static_cast<int>(threadIdx.x) + 128 * i) / PER_ROW;
            if (s >= s0 && s < s1) {
                uint32_t* w = &x[i].x;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t bad = __vcmpgtu2(w[e] & 0x7fff7fffu, kFinite);
                    w[e] |= bad & 0x7fff7fffu;
                    top = __vmaxu2(top, w[e] & ~bad & 0x7fff7fffu);
                }
            }
        }
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, m));
        __syncthreads();  // every warp has read the first maxima
        if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = top;
        __syncthreads();
        top = __vmaxu2(__vmaxu2(warp_max[0], warp_max[1]), __vmaxu2(warp_max[2], warp_max[3]));
    }
    const float2 tops = unpack2<BF16>(top);
    const float s_new = fmaxf(pow2_scale(fmaxf(tops.x, tops.y)), old);
    const float inv = s_new > 0.f ? 1.f / s_new : 0.f;  // exact
    if (threadIdx.x == 0) *scale = s_new;
    if (s0 > 0 && old < s_new) {  // the held codes move to the larger scale (from 0: they stand for zeros)
        const float ratio = old * inv;
        uint32_t* held = reinterpret_cast<uint32_t*>(codes);
        for (int i = threadIdx.x; i < s0 * (D / 4); i += 128) {
            const uint32_t v = held[i];
            uint32_t out = 0u;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const __half2_raw hr = __nv_cvt_fp8x2_to_halfraw2(
                    static_cast<__nv_fp8x2_storage_t>(v >> (16 * e)), __NV_E4M3);
                const float2 f = __half22float2(__half2(hr));
                out |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
                           make_float2(f.x * ratio, f.y * ratio), __NV_SATFINITE, __NV_E4M3))
                       << (16 * e);
            }
            held[i] = out;
        }
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
        const int c = static_cast<int>(threadIdx.x) + 128 * i, s = c / PER_ROW;
        if (s >= s0 && s < s1) {
            const uint32_t in[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            uint32_t out[2] = {0u, 0u};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = unpack2<BF16>(in[e]);
                out[e >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(
                                   make_float2(f.x * inv, f.y * inv), __NV_SATFINITE, __NV_E4M3))
                               << (16 * (e & 1));
            }
            reinterpret_cast<uint2*>(codes)[c] = make_uint2(out[0], out[1]);
        }
    }
}

struct AttendParams {
    const uint8_t* q;      // (B, Hq, T, D) 16-bit
    const uint8_t* codes[2];
    const float* scale[2];
    const int* table;      // (B, max_pages)
    const int* lens;       // tokens held, the queries' own included
    const int* q_lens;     // queries of each sequence; null: T
    uint8_t* o;
    float* lse;
    float* part;           // split sequences: (row, split, D) fp32, not normalised
    float2* part_ml;       // (row, split): maximum (log2 units) and sum
    int B, Hq, Hkv, T, num_pages, page_shift, max_pages;
    int mtiles;            // CTAs for the G T query rows of a key/value head
    int nsplit, split;     // splits of `split` tokens; the last takes what is left
    int causal;
    float scale_log2;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void* src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Two e4m3 codes (low half of v, or the high one) as two fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2(uint32_t v, bool high) {
    uint32_t r;
    const uint16_t h = static_cast<uint16_t>(high ? v >> 16 : v);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(h));
    return r;
}
// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), fp16; and the same from zero.
__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_from0(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// Transposes an 8 x 8 matrix of 16-bit values held as a fragment.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ void attend_lengths(const AttendParams& p, int b, int* len, int* tb, bool report) {
    const long long cap = static_cast<long long>(p.max_pages) << p.page_shift;
    int n = p.lens[b], t = p.q_lens ? p.q_lens[b] : p.T;
    if (n < 0 || n > cap || t < 0 || t > p.T) {
        if (report) record_bad_page();
        n = n < 0 ? 0 : (n > cap ? static_cast<int>(cap) : n);
        t = t < 0 ? 0 : (t > p.T ? p.T : t);
    }
    *len = n;
    *tb = t;
}

// One CTA per (8 NT query rows, split, key/value head, sequence); the G T rows of
// a key/value head (G query heads share it) are one matrix, so its codes are read
// once for up to 16 of them.  Four warps take 16-key tiles in turn, each with its
// own running maximum, sum and output, joined at the end.
//
// Both products run on fp16 tensor-core fragments (m16n8k16), transposed: S^T =
// K Q^T and O^T = V^T P^T, the query rows in the narrow (8) extent.  A single
// token is a handful of rows, far too few for the 128 of a tensor-memory tile,
// and what bounds the kernel is the codes' way from HBM and through the registers.
//   e4m3 converts to fp16 exactly.  q is brought into fp16 by a power of two for
// each row (its largest value in 8..16): exact down to 2^-18 of it.  P goes to
// fp16 rounded (half a step, 2^-11).  The running maximum of a row stays until a
// score exceeds it by more than 2^6 (all exponents and the final division use the
// same one), so P is at most 2^6; it is stored times 2^9, which leaves everything
// above 2^-23 of the maximum's weight in fp16's normal range.
//   The scale of K's page multiplies the scores in fp32.  O is kept in units of the
// largest scale u of V met so far: the scale s of a tile's page enters P as the
// factor s / u, or, below 2^-6, where P would leave fp16's range, the
// tile's own product in fp32.
//
// A fragment's K extent is a sum, in any order, so the lanes take features and
// keys in the order in which 16-byte pieces lie in memory: lane (g, t) (g = lane /
// 4, t = lane % 4) takes of K row g (and g + 8) features 16 t .. 16 t + 15 of each
// 64, and of V rows 2t, 2t+1, 2t+8, 2t+9 the features D/8 g .., a byte permute
// pairing two keys' codes.  Each lane thus reads, through shared memory, only what
// it copied itself (cp.async): no barrier but its own copies'.
//
// What bounds it: with 8 rows HBM and instruction latency at 16 warps an SM (128
// registers): 64 sequences of 2.7 to 8 thousand tokens, 8 key/value heads, d = 128:
// 155 us, 4.6 TB/s (5 CTAs an SM at 96 registers: 184; 3 at 150: 159; the query rows in
// the wide extent of the fragments, 16 of which a single token fills one: 239).  Few
// heads: the launch, four dependent loads and the join, about half of the time by estimate
// (no breakdown was taken): 16 heads of 4096 tokens 12.5 us.
// 16 rows convert the codes once for two fragments: 60 us for 16 x 2 heads of 16000
// tokens where 8 rows take 37.
template <int D, int NT>
struct AttendCfg {
    static constexpr int KP = D / 32, VP = 4;  // pieces of 16 keys: K 16 bytes each, V D/8 bytes
    static constexpr int VW = D / 32;          // words of a V piece
    static constexpr uint32_t V_OFF = KP * 512u, TILE = V_OFF + VP * 32u * (D / 8);
    static constexpr int STAGES = D == 128 ? (NT == 1 ? 3 : 4) : 6;
    static constexpr uint32_t WARP = STAGES * TILE;
    static constexpr int ROWS = 8 * NT, LD = D + 4;
    static constexpr uint32_t JOIN = 4 * ROWS * LD * 4 + 4 * ROWS * 8;
    static constexpr uint32_t SMEM = 4 * WARP > JOIN ? 4 * WARP : JOIN;
};

template <int D, bool BF16, int NT>
__global__ void __launch_bounds__(128, NT == 1 ? 4 : 3) cache_attend_kernel(const AttendParams p) {
    using C = AttendCfg<D, NT>;
    constexpr int ROWS = C::ROWS;
    constexpr float kRaise = 6.f, kUp = 9.f;  // log2 of P's bound and of its storage factor
    extern __shared__ __align__(16) uint8_t smem_raw[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    int id = blockIdx.x;
    const int mt = id % p.mtiles;
    id /= p.mtiles;
    const int split = id % p.nsplit;
    id /= p.nsplit;
    const int hk = id % p.Hkv, b = id / p.Hkv;
    int len, tb;
    attend_lengths(p, b, &len, &tb, threadIdx.x == 0);
    const int G = p.Hq / p.Hkv, rows = G * tb;  // row r: query r / G of head hk G + r % G
    const int k0 = split * p.split;
    if (mt * ROWS >= rows || (split > 0 && k0 >= len)) return;
    // keys past the last row's own position are seen by none of these rows
    const int seen = p.causal ? len - (tb - 1 - (min(rows, (mt + 1) * ROWS) - 1) / G) : len;
    const int k1 = min(seen, split == p.nsplit - 1 ? len : min(len, k0 + p.split));
    const bool whole = p.nsplit == 1 || len <= p.split;
    // --------------------------------------------- this warp's 16-key tiles
    // Step s is tile 4 s + warp; lane l looks up the page and scales of step l of 32
    // at a time, one batch ahead.
    const int tile0 = k0 >> 4, ntiles = k1 > k0 ? (k1 - k0 + 15) >> 4 : 0;  // splits start at tiles
    const int nsteps = (ntiles + 3 - warp) >> 2;              // of this warp
    auto look_up = [&](int batch, int& page, float& ks, float& vs) {
        const int step = batch * 32 + lane, tile = tile0 + 4 * step + warp;
        page = -1;
        ks = vs = 0.f;
        if (step < nsteps) {
            page = __ldg(p.table + static_cast<size_t>(b) * p.max_pages + (tile >> (p.page_shift - 4)));
            if (page < 0 || page >= p.num_pages) {
                record_bad_page();
                page = -1;
            } else {
                const size_t at = static_cast<size_t>(page) * p.Hkv + hk;
                ks = __ldg(p.scale[0] + at);
                vs = __ldg(p.scale[1] + at);
            }
        }
    };
    int page_a, page_b = -1;
    float ks_a, vs_a, ks_b = 0.f, vs_b = 0.f;
    look_up(0, page_a, ks_a, vs_a);
    if (nsteps > 32) look_up(1, page_b, ks_b, vs_b);
    uint8_t* const ring = smem_raw + warp * C::WARP;
    const uint8_t* const kbase = p.codes[0] + g * D + t4 * 16;
    const uint8_t* const vbase = p.codes[1] + 2 * t4 * D + g * (D / 8);
    const uint32_t kdst = smem_u32(ring) + lane * 16u, vdst = smem_u32(ring) + C::V_OFF + lane * (D / 8);
    int batch = 0;       // the batch that page_a holds
    int load_slot = 0;   // ring slot of the next load
    auto load = [&](int s) {
        if (s < nsteps) {
            const int page = __shfl_sync(0xffffffffu, (s >> 5) == batch ? page_a : page_b, s & 31);
            if (page >= 0) {
                const int slot = ((tile0 + 4 * s + warp) << 4) & ((1 << p.page_shift) - 1);
                const size_t at =
                    (((static_cast<size_t>(page) * p.Hkv + hk) << p.page_shift) + static_cast<size_t>(slot)) * D;
                const uint8_t* k = kbase + at;
#pragma unroll
                for (int i = 0; i < C::KP; ++i)  // keys g + 8 (i % 2), features 64 (i / 2) ..
                    cp_async16(kdst + load_slot * C::TILE + i * 512u, k + (i & 1) * 8 * D + (i >> 1) * 64);
                const uint8_t* v = vbase + at;
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // keys 2 t, 2 t + 1, 2 t + 8, 2 t + 9
                    const uint32_t d = vdst + load_slot * C::TILE + i * 4 * D;
                    const uint8_t* src = v + ((i & 1) + (i >> 1) * 8) * D;
                    if constexpr (D == 128) cp_async16(d, src); else cp_async8(d, src);
                }
            }
        }
        cp_async_commit();
        load_slot = load_slot == C::STAGES - 1 ? 0 : load_slot + 1;
    };
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s) load(s);
    // ------------------------------------------------------------ queries
    // B fragment of Q^T: row g of each 8, features as K's
    uint32_t qf[NT][D / 16][2];
    float up[NT];  // 2^k that brings the lane's row g into fp16
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        uint4 raw[D / 32];  // features 64 h + 16 t4 .. + 15
        const int r = mt * ROWS + n * 8 + g;
        uint32_t top = 0u;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            raw[c] = make_uint4(0u, 0u, 0u, 0u);
            if (r < rows) {
                const size_t row = (static_cast<size_t>(b) * p.Hq + hk * G + r % G) * p.T + r / G;
                raw[c] = __ldg(reinterpret_cast<const uint4*>(
                    p.q + (row * D + 64 * (c >> 1) + 16 * t4 + 8 * (c & 1)) * 2));
            }
            top = __vmaxu2(__vmaxu2(top, raw[c].x & 0x7fff7fffu), raw[c].y & 0x7fff7fffu);
            top = __vmaxu2(__vmaxu2(top, raw[c].z & 0x7fff7fffu), raw[c].w & 0x7fff7fffu);
        }
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float2 f = unpack2<BF16>(top);
        int e = 130 - static_cast<int>(__float_as_uint(fmaxf(f.x, f.y)) >> 23);
        e = e < -126 ? -126 : (e > 126 ? 126 : e);
        up[n] = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
            const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 x = unpack2<BF16>(w[j]);
                qf[n][2 * c + (j >> 1)][j & 1] = pack2<false>(x.x * up[n], x.y * up[n]);
            }
        }
    }
    // of this lane's result columns, rows 2 t and 2 t + 1 of each 8: the score
    // factor, the keys seen; and the keys that all rows see
    float mul[NT][2];
    int see[NT][2], all = len;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = mt * ROWS + n * 8 + 2 * t4 + i;
            mul[n][i] = p.scale_log2 / __shfl_sync(0xffffffffu, up[n], (2 * t4 + i) * 4);
            see[n][i] = r < rows ? (p.causal ? len - (tb - 1 - r / G) : len) : 0;
        }
    if (p.causal) all = len - (tb - 1 - mt * ROWS / G);
    if (all > k1) all = k1;
    float o[NT][D / 16][4];
    float m[NT][2], mb[NT][2], l[NT][2];  // maximum, the same as a base (0 for none), sum
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][j][e] = 0.f;
#pragma unroll
        for (int i = 0; i < 2; ++i) m[n][i] = -INFINITY, mb[n][i] = l[n][i] = 0.f;
    }
    float unit = 0.f;
    int slot = 0;
    for (int s = 0; s < nsteps; ++s) {
        const int page = __shfl_sync(0xffffffffu, page_a, s & 31);
        const float ks = __shfl_sync(0xffffffffu, ks_a, s & 31);
        const float vs = __shfl_sync(0xffffffffu, vs_a, s & 31);
        load(s + C::STAGES - 1);  // into the slot that the last step has read
        cp_async_wait<C::STAGES - 1>();
        const uint8_t* buf = ring + slot * C::TILE;
        slot = slot == C::STAGES - 1 ? 0 : slot + 1;
        const int key0 = (tile0 + 4 * s + warp) << 4;
        if (page >= 0) {
            // --------------------------------------------------- scores
            float x[NT][4];  // (key g, row 2t), (g, 2t + 1), (g + 8, 2t), (g + 8, 2t + 1)
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                const uint4 wa = *reinterpret_cast<const uint4*>(buf + (h * 2) * 512 + lane * 16);
                const uint4 wb = *reinterpret_cast<const uint4*>(buf + (h * 2 + 1) * 512 + lane * 16);
                const uint32_t a[4] = {wa.x, wa.y, wa.z, wa.w}, c[4] = {wb.x, wb.y, wb.z, wb.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t f[4] = {e4m3x2(a[j], false), e4m3x2(c[j], false), e4m3x2(a[j], true),
                                           e4m3x2(c[j], true)};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        if (h == 0 && j == 0)
                            mma_f16_from0(x[n], f, qf[n][0][0], qf[n][0][1]);
                        else
                            mma_f16(x[n], f, qf[n][h * 4 + j][0], qf[n][h * 4 + j][1]);
                    }
                }
            }
            bool raise = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) x[n][e] *= mul[n][e & 1] * ks;
            if (key0 + 16 > all) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = key0 + g + 8 * (e >> 1);
                        if (key >= see[n][e & 1] || key >= k1) x[n][e] = -INFINITY;
                    }
            }
            // -------------------------------------------------- softmax
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int i = 0; i < 2; ++i) raise |= fmaxf(x[n][i], x[n][i + 2]) > m[n][i] + kRaise;
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float v = fmaxf(fmaxf(x[n][i], x[n][i + 2]), m[n][i]);
#pragma unroll
                        for (int k = 4; k < 32; k <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, k));
                        const float base = v == -INFINITY ? 0.f : v, keep = ex2(m[n][i] - base);
                        m[n][i] = v;
                        mb[n][i] = base;
                        l[n][i] *= keep;
#pragma unroll
                        for (int j = 0; j < D / 16; ++j) o[n][j][i] *= keep, o[n][j][i + 2] *= keep;
                    }
            }
            if (vs > unit) {
                const float down = unit / vs;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int j = 0; j < D / 16; ++j)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[n][j][e] *= down;
                unit = vs;
            }
            const float ratio = unit > 0.f ? vs / unit : 0.f;
            const bool near = ratio >= 0.015625f;
            // P 2^9 s / u; the sums without s / u
            const float add = kUp + (near ? __log2f(ratio) : 0.f);
            const float back = near ? 1.f / ratio : 1.f;
            uint32_t pf[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float b0 = add - mb[n][0], b1 = add - mb[n][1];
                const float p0 = ex2(x[n][0] + b0), p1 = ex2(x[n][1] + b1), p2 = ex2(x[n][2] + b0),
                            p3 = ex2(x[n][3] + b1);
                l[n][0] = fmaf(p0 + p2, back, l[n][0]);
                l[n][1] = fmaf(p1 + p3, back, l[n][1]);
                pf[n][0] = transpose8x8(pack2<false>(p0, p1));
                pf[n][1] = transpose8x8(pack2<false>(p2, p3));
            }
            // ---------------------------------------------------- V^T P^T
            uint32_t vw[4][C::VW];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint8_t* src = buf + C::V_OFF + (i * 32 + lane) * (D / 8);
                if constexpr (D == 128) {
                    const uint4 w = *reinterpret_cast<const uint4*>(src);
                    vw[i][0] = w.x, vw[i][1] = w.y, vw[i][2] = w.z, vw[i][3] = w.w;
                } else {
                    const uint2 w = *reinterpret_cast<const uint2*>(src);
                    vw[i][0] = w.x, vw[i][1] = w.y;
                }
            }
            if (key0 + 16 > len) {  // slots past the last token may hold anything, NaN included
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (key0 + 2 * t4 + (i & 1) + (i >> 1) * 8 >= len) {
#pragma unroll
                        for (int w = 0; w < C::VW; ++w) vw[i][w] = 0u;
                    }
            }
#pragma unroll
            for (int w = 0; w < C::VW; ++w) {
                const uint32_t lo0 = __byte_perm(vw[0][w], vw[1][w], 0x5140),
                               hi0 = __byte_perm(vw[0][w], vw[1][w], 0x7362),
                               lo1 = __byte_perm(vw[2][w], vw[3][w], 0x5140),
                               hi1 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
                const uint32_t f0[4] = {e4m3x2(lo0, false), e4m3x2(lo0, true), e4m3x2(lo1, false),
                                        e4m3x2(lo1, true)};
                const uint32_t f1[4] = {e4m3x2(hi0, false), e4m3x2(hi0, true), e4m3x2(hi1, false),
                                        e4m3x2(hi1, true)};
                if (near) {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        mma_f16(o[n][2 * w], f0, pf[n][0], pf[n][1]);
                        mma_f16(o[n][2 * w + 1], f1, pf[n][0], pf[n][1]);
                    }
                } else {
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float own[2][4];
                        mma_f16_from0(own[0], f0, pf[n][0], pf[n][1]);
                        mma_f16_from0(own[1], f1, pf[n][0], pf[n][1]);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            o[n][2 * w][e] = fmaf(ratio, own[0][e], o[n][2 * w][e]);
                            o[n][2 * w + 1][e] = fmaf(ratio, own[1][e], o[n][2 * w + 1][e]);
                        }
                    }
                }
            }
        }
        if ((s & 31) == 31) {  // the next 32 steps
            ++batch;
            page_a = page_b, ks_a = ks_b, vs_a = vs_b;
            page_b = -1;
            if ((batch + 1) * 32 < nsteps) look_up(batch + 1, page_b, ks_b, vs_b);
        }
    }
    cp_async_wait<0>();
    cudaTriggerProgrammaticLaunchCompletion();
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 4; k < 32; k <<= 1) l[n][i] += __shfl_xor_sync(0xffffffffu, l[n][i], k);
    // ------------------------------------------------- the four warps' join
    __syncthreads();  // every warp is done with its ring
    constexpr int LD = C::LD;
    float* so = reinterpret_cast<float*>(smem_raw);                          // (warp, row, feature)
    float2* sml = reinterpret_cast<float2*>(smem_raw + 4 * ROWS * LD * 4);   // (warp, row)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int j = 0; j < D / 16; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float* dst = so + (warp * ROWS + n * 8 + 2 * t4 + i) * LD + g * (D / 8) + 2 * j;
                *reinterpret_cast<float2*>(dst) = make_float2(o[n][j][i] * unit, o[n][j][i + 2] * unit);
            }
        if (g == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                sml[warp * ROWS + n * 8 + 2 * t4 + i] = make_float2(m[n][i], l[n][i]);
        }
    }
    __syncthreads();
    constexpr int PER = 128 / ROWS;  // threads a row
    const int r = threadIdx.x / PER, c0 = threadIdx.x % PER;
    if (mt * ROWS + r >= rows) return;
    float mm = -INFINITY, ll = 0.f, f[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) mm = fmaxf(mm, sml[w * ROWS + r].x);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float2 ml = sml[w * ROWS + r];
        f[w] = ml.x == -INFINITY ? 0.f : ex2(ml.x - mm);
        ll += f[w] * ml.y;
    }
    const int rr = mt * ROWS + r;
    const size_t row = (static_cast<size_t>(b) * p.Hq + hk * G + rr % G) * p.T + rr / G;
    // both o and the sums carry P's storage factor: it leaves with the division,
    // and is taken out of the sum for the logarithm.  A sum is 0 only where no key was
    // seen; a NaN must not be taken for that.
    const float inv = whole ? (ll != 0.f ? 1.f / ll : 0.f) : 1.f;
#pragma unroll
    for (int c = c0 * 4; c < D; c += PER * 4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            const float4 a = *reinterpret_cast<const float4*>(so + (w * ROWS + r) * LD + c);
            v.x = fmaf(f[w], a.x, v.x), v.y = fmaf(f[w], a.y, v.y);
            v.z = fmaf(f[w], a.z, v.z), v.w = fmaf(f[w], a.w, v.w);
        }
        if (whole)
            *reinterpret_cast<uint2*>(p.o + (row * D + c) * 2) =
                make_uint2(pack2<BF16>(v.x * inv, v.y * inv), pack2<BF16>(v.z * inv, v.w * inv));
        else
            *reinterpret_cast<float4*>(p.part + (row * p.nsplit + split) * D + c) = v;
    }
    if (c0 == 0) {
        if (whole)
            p.lse[row] = ll != 0.f ? (mm + (log2f(ll) - kUp)) * 0.6931471805599453f : -INFINITY;
        else
            p.part_ml[row * p.nsplit + split] = make_float2(mm - kUp, ll);
    }
}

// Joins the splits of a row: one CTA a row, its warps taking splits in turn, lane l
// holding D / 32 features; the warps' sums meet in shared memory.  It is launched
// while the splits still run (programmatic dependent launch) and waits for them
// before it reads what they wrote.
template <int D, bool BF16>
__global__ void __launch_bounds__(256) cache_attend_join_kernel(const AttendParams p) {
    constexpr int E = D / 32, W = 8;
    __shared__ float so[W][D];
    __shared__ float sl[W];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row = blockIdx.x;
    const int t = static_cast<int>(row % p.T), b = static_cast<int>(row / p.T / p.Hq);
    int len, tb;
    attend_lengths(p, b, &len, &tb, false);  // inputs of both kernels
    cudaGridDependencySynchronize();         // every CTA: none ends before the splits have
    if (t >= tb || len <= p.split) return;   // no such query, or one split: stored already
    const int n = min(p.nsplit, (len + p.split - 1) / p.split);
    const float2* ml = p.part_ml + row * p.nsplit;
    const float* part = p.part + row * p.nsplit * D + lane * E;
    float mm = -INFINITY;
    for (int i = lane; i < n; i += 32) mm = fmaxf(mm, ml[i].x);
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, k));
    float acc[E], ll = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
#pragma unroll 8
    for (int i = warp; i < n; i += W) {
        const float2 v = ml[i];
        const float w = v.x == -INFINITY ? 0.f : ex2(v.x - mm);
        ll = fmaf(w, v.y, ll);
        float x[E];
        if constexpr (E == 4) {
            const float4 f = *reinterpret_cast<const float4*>(part + static_cast<size_t>(i) * D);
            x[0] = f.x, x[1] = f.y, x[2] = f.z, x[3] = f.w;
        } else {
            const float2 f = *reinterpret_cast<const float2*>(part + static_cast<size_t>(i) * D);
            x[0] = f.x, x[1] = f.y;
        }
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = fmaf(w, x[e], acc[e]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
    if (lane == 0) sl[warp] = ll;
    __syncthreads();
    if (threadIdx.x >= D / 2) return;
    float2 v = make_float2(0.f, 0.f);
    ll = 0.f;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        v.x += so[w][2 * threadIdx.x], v.y += so[w][2 * threadIdx.x + 1];
        ll += sl[w];
    }
    const float inv = ll != 0.f ? 1.f / ll : 0.f;
    reinterpret_cast<uint32_t*>(p.o)[row * (D / 2) + threadIdx.x] = pack2<BF16>(v.x * inv, v.y * inv);
    if (threadIdx.x == 0) p.lse[row] = ll != 0.f ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
}

// Rows of a CTA: 8, or 16 when there are more than 8 (the codes' conversion is
// then shared by two fragments of rows; with 24 or 40 rows a CTA, for 40 rows in
// all, 102 and 98 us against 94: fewer conversions, but fewer warps).
inline int attend_rows(int rows) { return rows > 8 ? 16 : 8; }

// Splits of a call whose sequences hold at most max_len tokens: four rounds of
// CTAs on the device's 148 multiprocessors (uneven lengths even out; the batch of 64
// takes 179, 174, 160, 155 and 155 us with one, two, three, four and six), but not
// below kLong tokens a split, then one round, but not below 256.
inline void attend_splits(int B, int Hkv, int mtiles, int max_len, int* nsplit, int* split) {
    constexpr long long kRound = 148 * 4, kLong = 1024, kShort = 256;
    const long long tokens = 1LL * B * Hkv * mtiles * max_len;
    long long len = tokens / (kRound * 4);
    if (len < kLong) {
        len = tokens / kRound;
        len = len > kLong ? kLong : (len < kShort ? kShort : len);
    }
    len = (len + 63) / 64 * 64;
    if (len > (1 << 30)) len = 1 << 30;
    *nsplit = static_cast<int>((max_len + len - 1) / len);
    *split = static_cast<int>(len);
}

}  // namespace attn
