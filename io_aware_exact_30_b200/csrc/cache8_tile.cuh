// Attention over the e4m3 cache for more than 16 query rows of a key/value head
// (several tokens, or many query heads that share it): tensor-memory tiles.
//
// One CTA per (64 query rows, split, key/value head, sequence) walks its keys in
// tiles of 128.  The codes are converted once for all rows:
//   K -> fp16, exactly; the page's scale multiplies the scores in fp32
//   V -> bf16, times the page's scale, exactly (4 significant bits, bf16 has fp32's
//        range: no page is too far from another)
//   Q -> fp16 by a power of two for each row, exact down to 2^-18 of its largest
// S = Q K^T and O += P V in tensor memory.  P goes to bf16 in two pieces (its rounding
// 2^-17), and the two pieces are two rows of one product: lanes 64-127 repeat the
// queries of lanes 0-63, make the same P and hand over its low piece, and O is the
// sum of the two lanes.
//
// bf16 has fp32's range, so P needs no running maximum to stay in bounds: a row's
// reference is the maximum of the first tile in which it sees a key, and one pass
// over S does a tile.  Only when a score exceeds the reference by more than 30 (log2: P
// up to 2^30, so that 2^31 terms of |v| <= 2^64 stay in fp32) is the reference moved
// and O rescaled.  Keys 0-63 and 64-127 of
// the tiles are two softmaxes of their own, each with its reference, sum and output,
// joined at the end: their warps never wait for one another.
//
// What bounds it: the softmax warps' chain (64 keys of a row a thread: about 2000
// cycles a tile, its exponentials alone 1000), which the lanes of the low pieces go
// through a second time, where the products take 1024 and a
// tile's 32 KB of codes 1400 of a multiprocessor's share of HBM; and 8 us before a CTA's
// first tile and after its last.  Measured: five queries of 8 heads a key/value head
// over 16 sequences of 5 to 16 thousand tokens, d = 128: 64 us (16-row fragments, which
// convert the codes three times: 94); 64 rows over 16000 tokens each: 68 us; 8192
// queries of 32 heads over themselves (8 key/value heads): 1.72 ms, 320 TFLOP/s.
//
// Roles (640 threads): warp 0 issues the products, warps 4-11 softmax (thread = lane;
// four warps a half of the keys) and output, warps 12-19 conversion: each 16 keys of
// a tile, which lie in one page; a lane reads back, through shared memory, the 16-byte
// pieces it copied itself (cp.async).  P is packed over the columns of S that its
// thread has read.
#pragma once

#include "cache8.cuh"
#include "ptx_more.cuh"

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
    static constexpr int B_KF = 0, B_VF = 2, B_SF = 4, B_OD = 6, B_PF = 8, B_QF = 10, B_XF = 11, B_DR = 12,
                         NBAR = 13;
    static constexpr uint32_t OFF_MISC = OFF_BAR + NBAR * 8;
    static constexpr uint32_t SMEM = OFF_MISC + 16 + 1024;
    static constexpr uint32_t COL_O = 256;  // S at 0 and 128, O of either half of the keys at 256 and 384
    static_assert(8u * RAW_WARP >= 64u * 2 * 8, "room for the halves' statistics");
    static_assert(SMEM <= 232448u, "dynamic shared memory above the sm_100 per-block limit");
};

template <int D, bool BF16>
__global__ void __launch_bounds__(640, 1) cache_attend_tile_kernel(const AttendParams p) {
    using C = AttendTileCfg<D>;
    constexpr float kRaise = 30.f;
    constexpr int ROWS = 64;
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
    if (mt * ROWS >= rows || (split > 0 && k0 >= len)) return;
    // keys past the last row's own position are seen by none of these rows
    const int seen = p.causal ? len - (tb - 1 - (min(rows, (mt + 1) * ROWS) - 1) / G) : len;
    const int k1 = min(seen, split == p.nsplit - 1 ? len : min(len, k0 + p.split));
    const bool whole = p.nsplit == 1 || len <= p.split;
    const int nt = k1 > k0 ? (k1 - k0 + 127) >> 7 : 0;
    const uint32_t bar0 = base + C::OFF_BAR;
#define ABAR(i) (bar0 + 8u * static_cast<uint32_t>(i))
    volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(gbase + C::OFF_MISC);
    volatile uint32_t* abort_flag = tmem_slot + 1;
    if (threadIdx.x == 0) {
        for (int i = 0; i < C::NBAR; ++i) {
            const bool all = i < C::B_SF || i == C::B_PF || i == C::B_PF + 1 || i == C::B_XF;
            mbar_init(ABAR(i), all ? 256 : (i == C::B_QF ? 128 : 1));
        }
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
    // registers of a thread by role; the launch gives each of the five warpgroups 96
    constexpr int R_ISSUE = 32, R_SOFT = 136, R_CONV = 80;
    static_assert(R_ISSUE + 2 * R_SOFT + 2 * R_CONV <= 5 * 96, "more registers than the launch has");
    if (warp < 4) {
        regs_down<R_ISSUE>();
    } else if (warp < 12) {
        regs_up<R_SOFT>();
    } else {
        regs_down<R_CONV>();
    }
    if (warp == 0) {
        // ------------------------------------------------------- MMA issuer
        if (elect_one()) {
            constexpr uint32_t ID_S = idesc_f16(false, 128, 128, false, false);  // Q K^T, fp16
            constexpr uint32_t ID_O = idesc_f16(true, 128, D, false, true);      // P V, bf16
            const uint64_t dq = sdesc_sw128(base, 16, 1024), dk = sdesc_sw128(base + C::OFF_K, 16, 1024),
                           dv = sdesc_sw128(base + C::OFF_V, 16384, 1024);
            constexpr uint32_t M16 = C::MAT >> 4;
            // S of tile j: its K written, its buffer (P of two tiles back) read by P V
            auto issue_s = [&](int j) -> bool {
                const int s = j & 1;
                if (!wait3(ABAR(C::B_KF + s), (j >> 1) & 1, true, ABAR(C::B_OD + s), ((j >> 1) - 1) & 1, j >= 2,
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
                if (!(ok = wait3(ABAR(C::B_PF + s), (j >> 1) & 1, true, ABAR(C::B_VF + s), (j >> 1) & 1, true, 0u, 0u,
                                 false, abort_flag)))
                    break;
                tc_fence_after();
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)  // 16 keys (2048 bytes) per step
                        mma_ts(tmem + C::COL_O + 128u * h, tmem + 128u * s + 64u * h + kk * 8u,
                               dv + s * M16 + (4 * h + kk) * 128u, ID_O, (j > 0 || kk > 0) ? 1u : 0u);
                mma_commit(ABAR(C::B_OD + s));
            }
            if (!ok) {
                mma_commit(ABAR(C::B_DR));
                wait_drain(ABAR(C::B_DR), 0);
            }
        }
        __syncwarp();
    } else if (warp >= 12) {
        // -------------------------------------------------------- conversion
        const int w = warp - 12;
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
        const int r = (warp & 3) * 32 + lane;       // TMEM lane
        const int hf = (warp - 4) >> 2;             // keys 64 hf.. of the tiles
        const bool low = (warp & 3) >= 2;           // the low pieces' lanes
        const int rr = mt * ROWS + (r & 63);
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const bool mine = mt * ROWS + (warp & 1) * 32 < rows;  // the warp has rows
        const size_t row = rr < rows
            ? (static_cast<size_t>(b) * p.Hq + hk * G + rr % G) * p.T + rr / G : 0;
        const int see = rr < rows ? min(k1, p.causal ? len - (tb - 1 - rr / G) : len) : 0;
        float mul;
        {
            // the row into fp16 by a power of two, rows past the last zero
            uint32_t top = 0u;
            const uint4* q = reinterpret_cast<const uint4*>(p.q + row * D * 2);
#pragma unroll
            for (int c = 0; c < D / 8; ++c) {
                const uint4 x = rr < rows ? __ldg(q + c) : make_uint4(0u, 0u, 0u, 0u);
                top = __vmaxu2(__vmaxu2(top, x.x & 0x7fff7fffu), x.y & 0x7fff7fffu);
                top = __vmaxu2(__vmaxu2(top, x.z & 0x7fff7fffu), x.w & 0x7fff7fffu);
            }
            const float2 f = unpack2<BF16>(top);
            int e = 130 - static_cast<int>(__float_as_uint(fmaxf(f.x, f.y)) >> 23);
            e = e < -126 ? -126 : (e > 126 ? 126 : e);
            const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
            mul = p.scale_log2 / up;
            if (hf == 0) {
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 v = rr < rows ? __ldg(q + c) : make_uint4(0u, 0u, 0u, 0u);
                    const uint32_t x[4] = {v.x, v.y, v.z, v.w};
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
        }
        const int all = __reduce_min_sync(0xffffffffu, rr < rows ? see : k1);  // keys all rows of the warp see
        float m = -INFINITY, mb = 0.f, l = 0.f;  // reference, the same as a base (0 for none), sum
        bool ok = true;
        for (int j = 0; j < nt; ++j) {
            const int s = j & 1, key0 = k0 + j * 128 + 64 * hf;
            if (!(ok = __all_sync(0xffffffffu, wait_bounded(ABAR(C::B_SF + s), (j >> 1) & 1, abort_flag)))) break;
            tc_fence_after();
            const uint32_t cols = lane_addr + 128u * s + 64u * hf;
            if (mine) {
                const float4 k4 = *reinterpret_cast<const float4*>(gbase + C::OFF_KS + (j & 3) * 32 + hf * 16);
                const float ks[4] = {k4.x, k4.y, k4.z, k4.w};
                const bool edge = key0 + 64 > all || k4.x < 0.f || k4.y < 0.f || k4.z < 0.f || k4.w < 0.f;
                uint32_t v[4][16];  // S of the 64 keys
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) tmem_ld16(cols + 16u * cc, v[cc]);
                tmem_ld_wait();
#pragma unroll
                for (int cc = 0; cc < 4; ++cc)
#pragma unroll
                    for (int e = 0; e < 16; ++e) reg_fence(v[cc][e]);
                // exponents against the reference
                const uint64_t minus = f2(-mb, -mb);
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) {
                    const float a = mul * ks[cc];
                    const uint64_t a2 = f2(a, a);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float2 y = unf2(fma2(f2(__uint_as_float(v[cc][2 * e]), __uint_as_float(v[cc][2 * e + 1])),
                                                   a2, minus));
                        v[cc][2 * e] = __float_as_uint(y.x), v[cc][2 * e + 1] = __float_as_uint(y.y);
                    }
                }
                if (edge) {
#pragma unroll
                    for (int cc = 0; cc < 4; ++cc) {
                        const int last = ks[cc] < 0.f ? 0 : see - (key0 + 16 * cc);  // keys seen of the 16
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            if (e >= last) v[cc][e] = __float_as_uint(-INFINITY);
                    }
                }
                float tops[4];
#pragma unroll
                for (int cc = 0; cc < 4; ++cc) {
                    tops[cc] = __uint_as_float(v[cc][0]);
#pragma unroll
                    for (int e = 1; e < 15; e += 2)
                        tops[cc] = max3(tops[cc], __uint_as_float(v[cc][e]), __uint_as_float(v[cc][e + 1]));
                    tops[cc] = fmaxf(tops[cc], __uint_as_float(v[cc][15]));
                }
                const float top = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]);
                // the row's first keys, or a score far above the reference
                const bool move = top > kRaise || (m == -INFINITY && top > -INFINITY);
                if (__any_sync(0xffffffffu, move)) {
                    // (what a first reference scales is still zero)
                    const float by = move ? top : 0.f, keep = m == -INFINITY ? 1.f : ex2(-by);
                    mb += by;
                    if (move) m = mb;
                    l *= keep;
                    if (j > 0) {  // O, once the last product is done
                        if (!(ok = __all_sync(0xffffffffu, wait_bounded(ABAR(C::B_OD + (s ^ 1)), ((j - 1) >> 1) & 1,
                                                                        abort_flag))))
                            break;
                        tc_fence_after();
#pragma unroll
                        for (int cc = 0; cc < D / 16; ++cc) {
                            uint32_t x[16];
                            tmem_ld16(lane_addr + C::COL_O + 128u * hf + 16u * cc, x);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                reg_fence(x[e]);
                                x[e] = __float_as_uint(__uint_as_float(x[e]) * keep);
                            }
                            tmem_st16(lane_addr + C::COL_O + 128u * hf + 16u * cc, x);
                        }
                    }
#pragma unroll
                    for (int cc = 0; cc < 4; ++cc)
#pragma unroll
                        for (int e = 0; e < 16; ++e) v[cc][e] = __float_as_uint(__uint_as_float(v[cc][e]) - by);
                }
                uint64_t sum = 0ull;
#pragma unroll
                for (int cc = 0; cc < 4; cc += 2) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        uint32_t &a = v[cc + (e >> 3)][2 * (e & 7)], &d = v[cc + (e >> 3)][2 * (e & 7) + 1];
                        const float pa = ex2(__uint_as_float(a)), pb = ex2(__uint_as_float(d));
                        sum = add2(sum, f2(pa, pb));
                        pk[e] = pack2<true>(pa, pb);
                        a = __float_as_uint(pa), d = __float_as_uint(pb);
                    }
                    if (low) {
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            const float2 f = unpack2<true>(pk[e]);
                            pk[e] = pack2<true>(__uint_as_float(v[cc + (e >> 3)][2 * (e & 7)]) - f.x,
                                                __uint_as_float(v[cc + (e >> 3)][2 * (e & 7) + 1]) - f.y);
                        }
                    }
                    tmem_st16(cols + 8u * cc, pk);
                }
                const float2 f = unf2(sum);
                l += f.x + f.y;
                tmem_st_wait();
            } else {  // lanes of rows past the last: P = 0
                uint32_t none[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) none[e] = 0u;
                tmem_st16(cols, none);
                tmem_st16(cols + 16u, none);
                tmem_st_wait();
            }
            tc_fence_before();
            mbar_arrive(ABAR(C::B_PF + s));
        }
        if (ok && nt > 0)
            ok = __all_sync(0xffffffffu, wait_bounded(ABAR(C::B_OD + ((nt - 1) & 1)), ((nt - 1) >> 1) & 1, abort_flag));
        tc_fence_after();
        // join: the four parts of a row (half of the keys, piece of P) through the
        // memory of K and V, which the products have read
        float* parts = reinterpret_cast<float*>(gbase + C::OFF_K);        // (part, feature, row)
        float2* ml = reinterpret_cast<float2*>(gbase + C::OFF_RAW);       // (half, row)
        if (ok) {
            float* x = parts + (hf * 2 + (low ? 1 : 0)) * D * 64 + (r & 63);
#pragma unroll
            for (int cc = 0; cc < D / 16; ++cc) {
                uint32_t v[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = 0u;
                if (nt > 0) {
                    tmem_ld16(lane_addr + C::COL_O + 128u * hf + 16u * cc, v);
                    tmem_ld_wait();
                }
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    reg_fence(v[e]);
                    x[(16 * cc + e) * 64] = __uint_as_float(v[e]);
                }
            }
            if (!low) ml[hf * 64 + (r & 63)] = make_float2(m, l);
            mbar_arrive(ABAR(C::B_XF));
            ok = __all_sync(0xffffffffu, wait_bounded(ABAR(C::B_XF), 0, abort_flag));
        }
        const int t = threadIdx.x - 128, q = t & 63, part = t >> 6, qq = mt * ROWS + q;
        if (ok && qq < rows) {
            const float2 a = ml[q], d = ml[64 + q];
            const float mm = fmaxf(a.x, d.x);
            const float fa = a.x == -INFINITY ? 0.f : ex2(a.x - mm), fd = d.x == -INFINITY ? 0.f : ex2(d.x - mm);
            const float ll = fa * a.y + fd * d.y;
            const float inv = whole ? (ll != 0.f ? 1.f / ll : 0.f) : 1.f;
            const size_t at = (static_cast<size_t>(b) * p.Hq + hk * G + qq % G) * p.T + qq / G;
#pragma unroll 4
            for (int c = part * (D / 4); c < (part + 1) * (D / 4); c += 4) {
                float v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float* x = parts + (c + e) * 64 + q;
                    // (a half whose row saw nothing holds zeros)
                    v[e] = (fa * (x[0] + x[D * 64]) + fd * (x[2 * D * 64] + x[3 * D * 64])) * inv;
                }
                if (whole)
                    *reinterpret_cast<uint2*>(p.o + (at * D + c) * 2) =
                        make_uint2(pack2<BF16>(v[0], v[1]), pack2<BF16>(v[2], v[3]));
                else
                    *reinterpret_cast<float4*>(p.part + (at * p.nsplit + split) * D + c) =
                        make_float4(v[0], v[1], v[2], v[3]);
            }
            if (part == 0) {
                if (whole)
                    p.lse[at] = ll != 0.f ? (mm + log2f(ll)) * 0.6931471805599453f : -INFINITY;
                else
                    p.part_ml[at * p.nsplit + split] = make_float2(mm, ll);
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

// How a call runs: tensor-memory tiles of 64 rows of a key/value head, or fragments
// of 8 or 16 rows a CTA; CTAs for its rows; splits.
struct AttendPlan {
    bool tiled;
    int rows, mtiles, nsplit, split;
};

// Tiles for more than 16 rows, of which a tile costs one as much as another: 24 rows
// over 16 x 2 heads of 16000 tokens take 62 us in tiles and 91 in fragments at d = 128
// (53 and 58 at d = 64), 16 rows 60 and 59 (52 and 37).  Up to 32 rows over few keys
// the fragments' shorter start counts: 32 rows over 8 heads of 4000 tokens 15.5 us
// against 17.3, over 4 x 2 heads of 500 tokens 12.6 against 15.1.
inline AttendPlan attend_plan(int B, int Hq, int Hkv, int T, int max_len) {
    AttendPlan p;
    if (max_len > (1 << 30)) max_len = 1 << 30;  // split * nsplit stays an int
    const int rows = Hq / Hkv * T;
    p.tiled = rows > 32 || (rows > 16 && 1LL * B * Hkv * max_len > (1 << 17));
    p.rows = p.tiled ? 64 : attend_rows(rows);
    p.mtiles = (rows + p.rows - 1) / p.rows;
    if (!p.tiled) {
        attend_splits(B, Hkv, p.mtiles, max_len, &p.nsplit, &p.split);
        return p;
    }
    // One CTA a multiprocessor.  One round of them where two splits or more fit into
    // it, else three (uneven lengths even out); splits of four tiles at least.
    const long long base = 1LL * B * Hkv * p.mtiles;
    long long n = 148 / base;
    if (n < 2) n = (3 * 148 + base - 1) / base;
    long long len = (max_len + n - 1) / n;
    len = (len + 127) / 128 * 128;
    if (len < 512) len = 512;
    if (len > (1 << 30)) len = 1 << 30;
    p.nsplit = static_cast<int>((max_len + len - 1) / len);
    p.split = static_cast<int>(len);
    return p;
}

inline size_t attend_workspace(int B, int Hq, int Hkv, int T, int D, int max_len) {
    const AttendPlan p = attend_plan(B, Hq, Hkv, T, max_len);
    return p.nsplit > 1 ? static_cast<size_t>(B) * Hq * T * p.nsplit * (D + 2) * 4 : 0;
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
void attend_launch(const AttendPlan& plan, const AttendParams& p, cudaStream_t st) {
    const unsigned grid = static_cast<unsigned>(p.mtiles) * p.nsplit * p.Hkv * p.B;
    if (plan.tiled)
        cache_attend_tile_kernel<D, BF16><<<grid, 640, AttendTileCfg<D>::SMEM, st>>>(p);
    else if (plan.rows == 8)
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
