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
// Bound by HBM for prompts (2 bytes read, 1 written per value) and by the
// launch for single tokens.
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
    const float2 tops = unpack2<BF16>(top);
    const float s_new = fmaxf(pow2_scale(fmaxf(tops.x, tops.y)), old);
    const float inv = s_new > 0.f ? 1.f / s_new : 0.f;  // exact
    if (threadIdx.x == 0) *scale = s_new;
    if (old > 0.f && old < s_new) {  // the held codes move to the larger scale
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
    int B, Hq, Hkv, T, num_pages, page, max_pages;
    int causal;
    float scale_log2;
};

// One warp per query row: keys one by one, the online softmax in every lane,
// lane l holding D / 32 features.
template <int D, bool BF16>
__global__ void __launch_bounds__(128) cache_attend_rows_kernel(const AttendParams p) {
    constexpr int E = D / 32;
    const long long row = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (row >= static_cast<long long>(p.B) * p.Hq * p.T) return;
    const int t = static_cast<int>(row % p.T);
    const int hq = static_cast<int>(row / p.T % p.Hq), b = static_cast<int>(row / p.T / p.Hq);
    const int hk = hq / (p.Hq / p.Hkv);
    const long long cap = static_cast<long long>(p.max_pages) * p.page;
    int len = p.lens[b], tb = p.q_lens ? p.q_lens[b] : p.T;
    if (len < 0 || len > cap || tb < 0 || tb > p.T) {
        if (lane == 0) record_bad_page();
        len = len < 0 ? 0 : (len > cap ? static_cast<int>(cap) : len);
        tb = tb < 0 ? 0 : (tb > p.T ? p.T : tb);
    }
    if (t >= tb) return;
    const int end = p.causal ? len - (tb - 1 - t) : len;
    float qv[E], acc[E];
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        const float2 f = unpack2<BF16>(*reinterpret_cast<const uint32_t*>(p.q + (row * D + lane * E + e) * 2));
        qv[e] = f.x, qv[e + 1] = f.y;
        acc[e] = acc[e + 1] = 0.f;
    }
    float m = -INFINITY, l = 0.f;
    for (int j = 0; j < end; ++j) {
        const int id_page = p.table[static_cast<size_t>(b) * p.max_pages + j / p.page];
        if (id_page < 0 || id_page >= p.num_pages) {
            if (lane == 0) record_bad_page();
            continue;
        }
        const size_t slot = static_cast<size_t>(id_page) * p.Hkv + hk;
        const size_t at = (slot * p.page + j % p.page) * D + lane * E;
        float kx[E], vx[E], dot = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            __nv_fp8_e4m3 c;
            c.__x = p.codes[0][at + e];
            kx[e] = static_cast<float>(c);
            c.__x = p.codes[1][at + e];
            vx[e] = static_cast<float>(c) * p.scale[1][slot];
            dot += qv[e] * kx[e];
        }
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, s);
        const float x = dot * p.scale[0][slot] * p.scale_log2;
        const float m2 = fmaxf(m, x), a = exp2f(m - m2), w = exp2f(x - m2);
        l = l * a + w;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * a + w * vx[e];
        m = m2;
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
#pragma unroll
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t*>(p.o + (row * D + lane * E + e) * 2) =
            pack2<BF16>(acc[e] * inv, acc[e + 1] * inv);
    if (lane == 0) p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace attn
