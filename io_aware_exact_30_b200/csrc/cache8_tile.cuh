// Attention over the e4m3 cache for more than 16 query rows of a key/value head
// (several tokens, or many query heads that share it): tensor-memory tiles.
//
// One CTA per (128 query rows, split, key/value head, sequence) walks its keys in
// tiles of 128.  The codes are converted once for all rows:
//   K -> fp16, exactly; the page's scale multiplies the scores in fp32
//   V -> bf16, times the page's scale, exactly (4 significant bits, bf16 has fp32's
//        range: no page is too far from another)
//   Q -> fp16 by a power of two for each row, exact down to 2^-18 of its largest
// S = Q K^T (tensor memory, two buffers), softmax with thread = row, P as two bf16
// pieces (its rounding 2^-17), O += P_hi V + P_lo V (tensor memory).  The kept maximum
// of a row moves when a score exceeds it by more than 2^6.
//
// Bound by HBM for up to 128 rows: 32 KB of codes a tile take 1400 cycles of a
// multiprocessor's share of bandwidth, the products about 1500 (S 512, P V twice 512),
// the conversion about 620 issue slots of each scheduler.
//
// Roles (512 threads): warp 0 issues the products, warps 4-7 softmax and output,
// warps 8-15 conversion: each 16 keys of a tile, which lie in one page; a lane
// reads back, through shared memory, the 16-byte pieces it copied itself (cp.async).
#pragma once

#include "cache8.cuh"

namespace attn {

template <int D>
struct AttendTileCfg {
    static constexpr uint32_t MAT = D * 256u;      // 128 rows of D 16-bit values
    static constexpr uint32_t OFF_K = MAT, OFF_V = 3 * MAT, OFF_RAW = 5 * MAT;
    static constexpr int PIECES = D / 32;          // 16-byte pieces of a lane: 16 keys of K (or V)
    static constexpr int STAGES = D == 128 ? 2 : 4;
    static constexpr uint32_t RAW_TILE = 2 * PIECES * 512u, RAW_WARP = STAGES * RAW_TILE;
    // K's scale of each 16 keys (< 0: no page) of four tiles: the softmax may still read
    // a tile's when the conversion is two tiles on
    static constexpr uint32_t OFF_KS = OFF_RAW + 8 * RAW_WARP;
    static constexpr uint32_t OFF_BAR = OFF_KS + 4 * 8 * 4;
    static constexpr int B_KF = 0, B_VF = 2, B_SF = 4, B_SR = 6, B_OD = 8, B_PF = 10, B_QF = 11, B_DR = 12,
                         NBAR = 13;
    static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr uint32_t SMEM = OFF_MISC + 16 + 1024;
    static constexpr uint32_t COL_P = 256, COL_O = 384;  // S at 0 and 128; P_hi, P_lo 64 columns each
    static_assert(SMEM <= 232448u, "dynamic shared memory above the sm_100 per-block limit");
};

template <int D, bool BF16>
__global__ void __launch_bounds__(512, 1) cache_attend_tile_kernel(const AttendParams p) {
    using C = AttendTileCfg<D>;
    constexpr float kRaise = 6.f;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw0 = smem_u32(smem_raw);
    const uint32_t base = (raw0 + 1023u) & ~1023u;
    uint8_t* gbase = smem_raw + (base - raw0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
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
    if (mt * 128 >= rows || (split > 0 && k0 >= len)) return;
    const int k1 = split == p.nsplit - 1 ? len : min(len, k0 + p.split);
    const bool whole = p.nsplit == 1 || len <= p.split;
    const int nt = k1 > k0 ? (k1 - k0 + 127) >> 7 : 0;
    const uint32_t bar0 = base + C::OFF_BAR;
#define ABAR(i) (bar0 + 8u * static_cast<uint32_t>(i))
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + C::OFF_MISC);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NBAR; ++i)
            mbar_init(ABAR(i), i < C::B_SF ? 256 : ((i >= C::B_SR && i < C::B_OD) || i == C::B_PF || i == C::B_QF ? 128 : 1));
        *abort_flag = 0u;
        fence_mbar_init();
    }
    if (warp == 0) {
        tmem_alloc(base + C::OFF_MISC, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (warp == 0) {
        // ------------------------------------------------------- MMA issuer
        uint32_t elected;
        asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(elected));
        if (elected) {
            constexpr uint32_t ID_S = idesc_f16(false, 128, 128, false, false);  // Q K^T, fp16
            constexpr uint32_t ID_O = idesc_f16(true, 128, D, false, true);      // P V, bf16
            const uint64_t dq = sdesc_sw128(base, 16, 1024), dk = sdesc_sw128(base + C::OFF_K, 16, 1024),
                           dv = sdesc_sw128(base + C::OFF_V, 16384, 1024);
            constexpr uint32_t M16 = C::MAT >> 4;
            // S of tile j: its K written, S's buffer read by the softmax two tiles back
            auto issue_s = [&](int j) -> bool {
                const int s = j & 1;
                if (!wait3(ABAR(C::B_KF + s), (j >> 1) & 1, true, ABAR(C::B_SR + s), ((j >> 1) - 1) & 1, j >= 2,
                           ABAR(C::B_QF), 0, j == 0, abort_flag))
                    return false;
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * 16384u + (kk & 3) * 32u) >> 4;
                    mma_ss(tmem + 128u * s, dq + off, dk + s * M16 + off, ID_S, kk > 0 ? 1u : 0u);
                }
                mma_commit(ABAR(C::B_SF + s));
                return true;
            };
            bool ok = nt == 0 || issue_s(0);
            for (int j = 0; ok && j < nt; ++j) {
                const int s = j & 1;
                if (j + 1 < nt && !(ok = issue_s(j + 1))) break;
                if (!(ok = wait3(ABAR(C::B_PF), j & 1, true, ABAR(C::B_VF + s), (j >> 1) & 1, true, 0u, 0u, false,
                                 abort_flag)))
                    break;
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int kk = 0; kk < 8; ++kk)  // 16 keys (2048 bytes) per step
                        mma_ts(tmem + C::COL_O, tmem + C::COL_P + 64u * h + kk * 8u, dv + s * M16 + kk * 128u, ID_O,
                               (j > 0 || h > 0 || kk > 0) ? 1u : 0u);
                mma_commit(ABAR(C::B_OD + s));
            }
            if (!ok) {
                mma_commit(ABAR(C::B_DR));
                wait_drain(ABAR(C::B_DR), 0);
            }
        }
        __syncwarp();
    } else if (warp >= 8) {
        // -------------------------------------------------------- conversion
        const int w = warp - 8;
        const int nw = k1 > k0 + 16 * w ? (k1 - k0 - 16 * w + 127) >> 7 : 0;  // tiles with keys of this warp
        // lane l looks up the page and scales of tile l of 32 at a time, one batch ahead
        auto look_up = [&](int batch, int& page, float& ks, float& vs) {
            const int tile = batch * 32 + lane;
            page = -1;
            ks = vs = 0.f;
            if (tile < nw) {
                page = __ldg(p.table + static_cast<size_t>(b) * p.max_pages +
                             ((k0 + tile * 128 + 16 * w) >> p.page_shift));
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
        int page_a, page_b = -1, batch = 0;
        float ks_a, vs_a, ks_b = 0.f, vs_b = 0.f;
        look_up(0, page_a, ks_a, vs_a);
        if (nt > 32) look_up(1, page_b, ks_b, vs_b);
        // piece i of a lane: key i PER + lane / LPR, 16 features from 16 (lane % LPR)
        constexpr int LPR = D / 16, PER = 32 / LPR;
        const int key0 = lane / LPR, c = lane % LPR;
        uint8_t* const ring = gbase + C::OFF_RAW + w * C::RAW_WARP + lane * 16;
        const uint32_t ring_at = smem_u32(ring);
        auto load = [&](int j) {
            if (j < nt) {
                const int page = __shfl_sync(0xffffffffu, (j >> 5) == batch ? page_a : page_b, j & 31);
                if (page >= 0) {
                    const int slot = (k0 + j * 128 + 16 * w) & ((1 << p.page_shift) - 1);
                    const size_t at = (((static_cast<size_t>(page) * p.Hkv + hk) << p.page_shift) +
                                       static_cast<size_t>(slot + key0)) * D + c * 16;
                    const uint32_t dst = ring_at + (j % C::STAGES) * C::RAW_TILE;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv)
#pragma unroll
                        for (int i = 0; i < C::PIECES; ++i)
                            cp_async16(dst + (kv * C::PIECES + i) * 512u, p.codes[kv] + at + i * PER * D);
                }
            }
            cp_async_commit();
        };
#pragma unroll
        for (int j = 0; j < C::STAGES; ++j) load(j);
        // 16-byte piece e of this lane's features of key k: of the atom of 64 features
        // c / 4, pieces 2 (c % 4) and the next; lanes of the second atom start with
        // the second, so that a row's lanes meet no bank twice
        auto place = [&](uint32_t mat, int key, int e) -> uint4* {
            return reinterpret_cast<uint4*>(gbase + mat + (c >> 2) * 16384u + key * 128 +
                                            (((2 * (c & 3) + e) ^ (key & 7)) << 4));
        };
        for (int j = 0; j < nt; ++j) {
            const int s = j & 1;
            const int page = __shfl_sync(0xffffffffu, page_a, j & 31);
            const float ks = __shfl_sync(0xffffffffu, ks_a, j & 31), vs = __shfl_sync(0xffffffffu, vs_a, j & 31);
            cp_async_wait<C::STAGES - 1>();
            const uint8_t* src = ring + (j % C::STAGES) * C::RAW_TILE;
            // K: its buffer was read by S of two tiles back
            if (j >= 2 && !__all_sync(0xffffffffu, wait_bounded(ABAR(C::B_SF + s), ((j >> 1) - 1) & 1, abort_flag)))
                break;
            if (lane == 0) *reinterpret_cast<float*>(gbase + C::OFF_KS + ((j & 3) * 8 + w) * 4) = page >= 0 ? ks : -1.f;
#pragma unroll
            for (int i = 0; i < C::PIECES; ++i) {
                const uint4 v = *reinterpret_cast<const uint4*>(src + i * 512);
                const uint32_t x[4] = {v.x, v.y, v.z, v.w};
                uint32_t h[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) h[2 * e] = e4m3x2(x[e], false), h[2 * e + 1] = e4m3x2(x[e], true);
                const int key = 16 * w + i * PER + key0, sw = (c >> 2) & 1;
                const uint4 a = make_uint4(h[0], h[1], h[2], h[3]), d = make_uint4(h[4], h[5], h[6], h[7]);
                *place(C::OFF_K + s * C::MAT, key, sw) = sw ? d : a;
                *place(C::OFF_K + s * C::MAT, key, sw ^ 1) = sw ? a : d;
            }
            fence_proxy_async_smem();
            mbar_arrive(ABAR(C::B_KF + s));
            // V: its buffer was read by P V of two tiles back
            if (j >= 2 && !__all_sync(0xffffffffu, wait_bounded(ABAR(C::B_OD + s), ((j >> 1) - 1) & 1, abort_flag)))
                break;
#pragma unroll
            for (int i = 0; i < C::PIECES; ++i) {
                const int key = 16 * w + i * PER + key0, sw = (c >> 2) & 1;
                uint32_t h[8];
                // slots that hold no token of this sequence may hold anything, NaN included
                const bool live = page >= 0 && k0 + j * 128 + key < k1;
                const uint4 v = *reinterpret_cast<const uint4*>(src + (C::PIECES + i) * 512);
                const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float2 f = unpack2<false>(e4m3x2(x[e >> 1], (e & 1) != 0));
                    h[e] = live ? pack2<true>(f.x * vs, f.y * vs) : 0u;
                }
                const uint4 a = make_uint4(h[0], h[1], h[2], h[3]), d = make_uint4(h[4], h[5], h[6], h[7]);
                *place(C::OFF_V + s * C::MAT, key, sw) = sw ? d : a;
                *place(C::OFF_V + s * C::MAT, key, sw ^ 1) = sw ? a : d;
            }
            fence_proxy_async_smem();
            mbar_arrive(ABAR(C::B_VF + s));
            load(j + C::STAGES);  // into the slot just read
            if ((j & 31) == 31) {
                ++batch;
                page_a = page_b, ks_a = ks_b, vs_a = vs_b;
                page_b = -1;
                if ((batch + 1) * 32 < nt) look_up(batch + 1, page_b, ks_b, vs_b);
            }
        }
        cp_async_wait<0>();
    } else if (warp >= 4) {
        // ------------------------------------------------ softmax and output
        const int r = (warp & 3) * 32 + lane, rr = mt * 128 + r;  // row == TMEM lane
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const bool mine = mt * 128 + (warp & 3) * 32 < rows;  // the warp has rows
        const size_t row = rr < rows
            ? (static_cast<size_t>(b) * p.Hq + hk * G + rr % G) * p.T + rr / G : 0;
        float mul = 0.f;
        int see = 0;
        {
            // the row into fp16 by a power of two, rows past the last zero
            uint4 q[D / 8];
            uint32_t top = 0u;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                q[c] = make_uint4(0u, 0u, 0u, 0u);
                if (rr < rows) q[c] = __ldg(reinterpret_cast<const uint4*>(p.q + row * D * 2) + c);
                top = __vmaxu2(__vmaxu2(top, q[c].x & 0x7fff7fffu), q[c].y & 0x7fff7fffu);
                top = __vmaxu2(__vmaxu2(top, q[c].z & 0x7fff7fffu), q[c].w & 0x7fff7fffu);
            }
            const float2 f = unpack2<BF16>(top);
            int e = 130 - static_cast<int>(__float_as_uint(fmaxf(f.x, f.y)) >> 23);
            e = e < -126 ? -126 : (e > 126 ? 126 : e);
            const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
            mul = p.scale_log2 / up;
            if (rr < rows) see = p.causal ? len - (tb - 1 - rr / G) : len;
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                const uint32_t x[4] = {q[c].x, q[c].y, q[c].z, q[c].w};
                uint32_t h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const float2 y = unpack2<BF16>(x[k]);
                    h[k] = pack2<false>(y.x * up, y.y * up);
                }
                *reinterpret_cast<uint4*>(gbase + (c >> 3) * 16384u + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
                    make_uint4(h[0], h[1], h[2], h[3]);
            }
            fence_proxy_async_smem();
            mbar_arrive(ABAR(C::B_QF));
        }
        if (see > k1) see = k1;
        const int all = __reduce_min_sync(0xffffffffu, rr < rows ? see : k1);  // keys all rows of the warp see
        float m = -INFINITY, mb = 0.f, l = 0.f;
        bool ok = true;
        for (int j = 0; j < nt; ++j) {
            const int s = j & 1, key0 = k0 + j * 128;
            if (!(ok = __all_sync(0xffffffffu, wait_bounded(ABAR(C::B_SF + s), (j >> 1) & 1, abort_flag)))) break;
            tc_fence_after();
            float4 ks4[2] = {*reinterpret_cast<const float4*>(gbase + C::OFF_KS + (j & 3) * 32),
                             *reinterpret_cast<const float4*>(gbase + C::OFF_KS + (j & 3) * 32 + 16)};
            const float ks[8] = {ks4[0].x, ks4[0].y, ks4[0].z, ks4[0].w, ks4[1].x, ks4[1].y, ks4[1].z, ks4[1].w};
            bool edge = key0 + 128 > all;
#pragma unroll
            for (int g = 0; g < 8; ++g) edge |= ks[g] < 0.f;
            // scores of 32 keys (two pages' worth of 16), log2 units
            auto scores = [&](int cc, float (&x)[32]) {
                uint32_t v[32];
                tmem_ld32(lane_addr + 128u * s + 32u * cc, v);
                tmem_ld_wait();
                reg_fence32(v);
                const float a = mul * ks[2 * cc], d = mul * ks[2 * cc + 1];
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(v[e]) * (e < 16 ? a : d);
                if (edge) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (ks[2 * cc + (e >> 4)] < 0.f || key0 + 32 * cc + e >= see) x[e] = -INFINITY;
                }
            };
            float top = -INFINITY;
            if (mine) {
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) {
                    float x[32];
                    scores(cc, x);
#pragma unroll
                    for (int e = 0; e < 32; e += 2) top = max3(top, x[e], x[e + 1]);
                }
            }
            // P's and O's last product is done: both may be written
            if (j > 0 && !(ok = __all_sync(0xffffffffu, wait_bounded(ABAR(C::B_OD + (s ^ 1)), ((j - 1) >> 1) & 1, abort_flag))))
                break;
            tc_fence_after();
            if (mine) {
                if (__any_sync(0xffffffffu, top > m + kRaise)) {
                    const float up = fmaxf(top, m);
                    const float next = up == -INFINITY ? 0.f : up, keep = ex2(m - next);
                    m = up, mb = next, l *= keep;
                    if (j > 0) {
#pragma unroll
                        for (int cc = 0; cc < D / 32; ++cc) {
                            uint32_t v[32];
                            tmem_ld32(lane_addr + C::COL_O + 32u * cc, v);
                            tmem_ld_wait();
                            reg_fence32(v);
#pragma unroll
                            for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * keep);
                            tmem_st32(lane_addr + C::COL_O + 32u * cc, v);
                        }
                    }
                }
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) {
                    float x[32];
                    scores(cc, x);
                    uint32_t hi[16], lo[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float a = ex2(x[2 * e] - mb), d = ex2(x[2 * e + 1] - mb);
                        l += a + d;
                        hi[e] = pack2<true>(a, d);
                        const float2 f = unpack2<true>(hi[e]);
                        lo[e] = pack2<true>(a - f.x, d - f.y);
                    }
                    tmem_st16(lane_addr + C::COL_P + 16u * cc, hi);
                    tmem_st16(lane_addr + C::COL_P + 64u + 16u * cc, lo);
                }
                tmem_st_wait();
            } else if (j == 0) {  // rows past the last: P stays zero
                uint32_t none[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) none[e] = 0u;
#pragma unroll
                for (int cc = 0; cc < 8; ++cc) tmem_st16(lane_addr + C::COL_P + 16u * cc, none);
                tmem_st_wait();
            }
            tc_fence_before();
            mbar_arrive(ABAR(C::B_SR + s));
            mbar_arrive(ABAR(C::B_PF));
        }
        if (ok && nt > 0)
            ok = __all_sync(0xffffffffu, wait_bounded(ABAR(C::B_OD + ((nt - 1) & 1)), ((nt - 1) >> 1) & 1, abort_flag));
        tc_fence_after();
        if (ok && mine) {
            const float inv = whole ? (l > 0.f ? 1.f / l : 0.f) : 1.f;
#pragma unroll
            for (int cc = 0; cc < D / 32; ++cc) {
                uint32_t v[32];
                if (nt > 0) {
                    tmem_ld32(lane_addr + C::COL_O + 32u * cc, v);
                    tmem_ld_wait();
                    reg_fence32(v);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) v[e] = 0u;
                }
                if (rr < rows) {
                    if (whole) {
                        uint4* dst = reinterpret_cast<uint4*>(p.o + (row * D + 32 * cc) * 2);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            uint32_t h[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                h[k] = pack2<BF16>(__uint_as_float(v[8 * e + 2 * k]) * inv,
                                                   __uint_as_float(v[8 * e + 2 * k + 1]) * inv);
                            dst[e] = make_uint4(h[0], h[1], h[2], h[3]);
                        }
                    } else {
                        float4* dst = reinterpret_cast<float4*>(p.part + (row * p.nsplit + split) * D + 32 * cc);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            dst[e] = make_float4(__uint_as_float(v[4 * e]), __uint_as_float(v[4 * e + 1]),
                                                 __uint_as_float(v[4 * e + 2]), __uint_as_float(v[4 * e + 3]));
                    }
                }
            }
            if (rr < rows) {
                if (whole)
                    p.lse[row] = l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
                else
                    p.part_ml[row * p.nsplit + split] = make_float2(m, l);
            }
        }
    }
#undef ABAR
    tc_fence_before();
    __syncthreads();
    cudaTriggerProgrammaticLaunchCompletion();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Which form a call takes: fragments for up to 16 rows of a key/value head, tiles
// for more.
inline bool attend_tiled(int Hq, int Hkv, int T) { return Hq / Hkv * T > 16; }
inline int attend_ctas(int Hq, int Hkv, int T) {
    return attend_tiled(Hq, Hkv, T) ? (Hq / Hkv * T + 127) / 128 : attend_mtiles(Hq, Hkv, T);
}
inline void attend_plan(int B, int Hq, int Hkv, int T, int max_len, int* nsplit, int* split) {
    const int mtiles = attend_ctas(Hq, Hkv, T);
    if (!attend_tiled(Hq, Hkv, T)) return attend_splits(B, Hkv, mtiles, max_len, nsplit, split);
    // two rounds of one CTA a multiprocessor, splits of four tiles at least
    if (max_len > (1 << 30)) max_len = 1 << 30;
    long long len = 1LL * B * Hkv * mtiles * max_len / (148 * 2);
    len = (len + 127) / 128 * 128;
    if (len < 512) len = 512;
    if (len > (1 << 30)) len = 1 << 30;
    *nsplit = static_cast<int>((max_len + len - 1) / len);
    *split = static_cast<int>(len);
}

inline size_t attend_workspace(int B, int Hq, int Hkv, int T, int D, int max_len) {
    int nsplit, split;
    attend_plan(B, Hq, Hkv, T, max_len, &nsplit, &split);
    return nsplit > 1 ? static_cast<size_t>(B) * Hq * T * nsplit * (D + 2) * 4 : 0;
}

template <int D, bool BF16>
bool attend_set_attributes() {
    return cudaFuncSetAttribute(cache_attend_kernel<D, BF16, 1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(AttendCfg<D, 1>::SMEM)) == cudaSuccess &&
           cudaFuncSetAttribute(cache_attend_kernel<D, BF16, 2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(AttendCfg<D, 2>::SMEM)) == cudaSuccess &&
           cudaFuncSetAttribute(cache_attend_tile_kernel<D, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                static_cast<int>(AttendTileCfg<D>::SMEM)) == cudaSuccess;
}

template <int D, bool BF16>
void attend_launch(const AttendParams& p, cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>(p.mtiles) * p.nsplit * p.Hkv * p.B;
    if (attend_tiled(p.Hq, p.Hkv, p.T))
        cache_attend_tile_kernel<D, BF16><<<grid, 512, AttendTileCfg<D>::SMEM, st>>>(p);
    else if (attend_rows(p.Hq, p.Hkv, p.T) == 8)
        cache_attend_kernel<D, BF16, 1><<<grid, 128, AttendCfg<D, 1>::SMEM, st>>>(p);
    else
        cache_attend_kernel<D, BF16, 2><<<grid, 128, AttendCfg<D, 2>::SMEM, st>>>(p);
    if (p.nsplit > 1) {
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(static_cast<unsigned>(p.B) * p.Hq * p.T);
        cfg.blockDim = dim3(256);
        cfg.stream = st;
        cudaLaunchAttribute early;
        early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
        early.val.programmaticStreamSerializationAllowed = 1;
        cfg.attrs = &early;
        cfg.numAttrs = 1;
        cudaLaunchKernelEx(&cfg, cache_attend_join_kernel<D, BF16>, p);
    }
}

}  // namespace attn
