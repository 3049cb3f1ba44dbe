// Attention mass of a batch's query rows (bf16 pools) on tcgen05 / TMEM:
//     mass[n] = sum over rows i of 2^(s_in - M_i) / L_i,   L_i = sum over n of 2^(s_in - M_i)
// with s the scores in the log2 domain. L_i is not known before all of row i's
// scores are, and keeping the scores takes more memory time than forming them again (a 128 x 128
// tile of them is 64 KB to write and to read, 2.9 us of an SM's share of the bandwidth; its MMAs
// take 0.8 us), so there are two passes over the keys and a reduction:
//   pass 1  running maximum and sum of each row (thread = row)
//   pass 2  the rows' weights, summed per key: one float per key and block of 128
//           rows goes to the workspace
//   reduce  the row blocks' floats in order, plus decay * mass_in
// No atomics: equal calls give equal bits.
//
// The scores are held to fp32 accuracy: a rotated q or k in one fp16 number would
// be off by up to 2^-11, about 3e-4 on a weight. Each goes in as hi + lo (lo: the rounding of
// the rest; lo's own steps end at 2^-24, so a component below 1/8 is exact to 2^-25 and not to 2^-22 of
// itself), and the accumulator takes K_lo Q_hi, K_hi Q_lo, then K_hi Q_hi, small
// ones first. That is 24 MMAs of 128 x 128 x 16 per 128 x 128 scores, and what bounds both passes.
//
// CTA = (request, KV head, two blocks of 128 rows = (token, head of the group) pairs, share
// of the tiles of 128 keys). Q is the MMAs' A operand in tensor memory: an MMA then
// reads 4 KB of shared memory in its 64 cycles, not 8 (which is all that
// the shared memory gives, with the rotation's own traffic on top), and the space goes to a third K
// stage. Roles (20 warps):
//   warp 0        producer: block table, TMA of K pages and of their position-table rows
//   warp 1        TMEM owner, MMA issuer
//   warps 4-11    two warpgroups. Two row blocks: each builds its own block's Q and takes its
//                 scores of every tile. One: they take the tiles of the one block in turn
//   warps 12-19   rotation: thread = (page, half of its slots, 4 frequencies), bf16 in
//                 place to hi, lo beside it
// Column sums of pass 2: TMEM is read in the fragment layout, where a thread holds 4 rows of
// the same 8 columns; it adds those, 7 shuffles join the 8 threads of a column, and the
// four warps meet in shared memory. Every wait is bounded, as in the prefill kernel.
//
// Measured (GB300): 8 requests of ~17,400 keys, 100..128 rows, 32/8 heads: 713-718 us, of which
// the MMAs are 430 (67 cycles each) and the rest the issuer's gaps between tiles (~500
// cycles) and the roles' contention: without the threads' arithmetic on the scores a pass takes
// 298 us of its 343, without the rotation 291. 16 requests of 2,112 keys, 64 rows: 106 us,
// where the ~8 us before a CTA's first MMA count too. Not kept: N = 64 MMAs (as slow as N = 128
// with A in tensor memory), two issuing warps (both S buffers finish together and the pipe
// waits for the arithmetic), all eight warps on each buffer in turn (pass 2 slower by a tenth).
#include <limits.h>

#include <type_traits>

#include "internal.h"
#include "tc_ptx.cuh"

namespace lazyattn {

namespace {

using namespace tc;

constexpr int kD = 128;
constexpr int kTileM = 128;                        // rows per block; two blocks per CTA
constexpr int kN = 128;                            // keys per tile
constexpr int kPagesPerTile = kN / kPage;          // 8
constexpr int kStages = 3;
constexpr int kInfoSlots = 8;                      // the scores of tile k - 8 were read before tile k's copies start
constexpr int kThreads = 640;
constexpr int kHalf = kTileM * 128;                // 16 KB: 64 dims of 128 rows or keys
constexpr int kTile = 2 * kHalf;                   // 32 KB: one fp16 operand tile
constexpr int kBaseBytes = kPagesPerTile * 512;    // 8 position-table rows
constexpr int kOffK = 0;                           // stages of (K hi, K lo)
constexpr int kOffBase = kOffK + kStages * 2 * kTile;
constexpr int kOffSum = kOffBase + kStages * kBaseBytes;   // pass 2: [warpgroup][tile parity][warp][key] column sums
constexpr int kSmemBytes = kOffSum + 2 * 2 * 4 * kN * 4 + 1024;
constexpr uint32_t kTmemCols = 512;                // S buffers of 128 columns; from 256 on Q hi, Q lo (64 each) of both blocks
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleThreshold = 8.0f;          // log2 units
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

struct TileInfo {
    int j;                        // tile index, -1: no more tiles
    int start[kPagesPerTile];     // logical position of slot 0 of each page
    int n[kPagesPerTile];         // keys in each page
    int full_from;                // every page full: rows at positions >= this see every key; else INT_MAX
};

struct MassParams {
    const uint64_t* entries;
    const int32_t* entry_offsets;
    const int32_t* entry_delta;   // doc-local pools
    const int32_t* q_offsets;
    const int32_t* q_start;
    const __nv_bfloat16* q;
    int32_t total_q, max_rows;    // max_rows: query tokens per request (host bound)
    int32_t g;
    int32_t oob_row;
    int32_t row_blocks;           // rows of the position table's 16-row view
    int32_t blocks;               // row blocks per request (host bound), an even number
    int32_t splits;
    int32_t cap;                  // entries per request (host bound)
    int32_t requests;
    float2* stats;                // [r][h][block][split][2][128] (reference maximum, sum)
    float* sums;                  // [block][r][cap][Hkv][16]
};

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
}
// Two fp32 lanes per instruction (packed f32x2 arithmetic).
__device__ __forceinline__ uint64_t pack2(float2 a) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a.x), "f"(a.y));
    return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t r) {
    float2 o;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(o.x), "=f"(o.y) : "l"(r));
    return o;
}
__device__ __forceinline__ float2 f2_mul(float2 a, float2 b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)));
    return unpack2(r);
}
__device__ __forceinline__ float2 f2_add(float2 a, float2 b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)));
    return unpack2(r);
}
__device__ __forceinline__ float2 f2_sub(float2 a, float2 b) {
    uint64_t r;
    asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)));
    return unpack2(r);
}
__device__ __forceinline__ float2 f2_fma(float2 a, float2 b, float2 c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(pack2(a)), "l"(pack2(b)), "l"(pack2(c)));
    return unpack2(r);
}
// What the fp16 pair `hi` leaves of (a, b), rounded to fp16.
__device__ __forceinline__ uint32_t rest_h2(float a, float b, uint32_t hi) {
    const float2 f = f2_sub(make_float2(a, b), __half22float2(*reinterpret_cast<const __half2*>(&hi)));
    return pack_h2(f.x, f.y);
}
__device__ __forceinline__ float bf_lo(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float bf_hi(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[8]) {
    x[0] = bf_lo(v.x); x[1] = bf_hi(v.x); x[2] = bf_lo(v.y); x[3] = bf_hi(v.y);
    x[4] = bf_lo(v.z); x[5] = bf_hi(v.z); x[6] = bf_lo(v.w); x[7] = bf_hi(v.w);
}
__device__ __forceinline__ void split8(const float (&x)[8], uint4& hi, uint4& lo) {
    hi = make_uint4(pack_h2(x[0], x[1]), pack_h2(x[2], x[3]), pack_h2(x[4], x[5]), pack_h2(x[6], x[7]));
    lo = make_uint4(rest_h2(x[0], x[1], hi.x), rest_h2(x[2], x[3], hi.y), rest_h2(x[4], x[5], hi.z),
                    rest_h2(x[6], x[7], hi.w));
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Page in range and positions inside the table: number of keys, 0 if none, -1 if unusable.
__device__ __forceinline__ int usable_tokens(const PoolView& pv, uint64_t e) {
    const int n = entry_nvalid(e);
    if (n == 0) return 0;
    if (entry_page(e) >= (uint32_t)pv.num_pages || n > kPage || entry_start(e) + n > pv.max_position) return -1;
    return n;
}
__device__ __forceinline__ int usable_local(const PoolView& pv, uint64_t e, int delta) {
    const int n = usable_tokens(pv, e);
    return n > 0 && (delta < 0 || delta > entry_start(e) || delta >= pv.max_position) ? -1 : n;
}

__device__ __forceinline__ size_t stats_at(const MassParams& P, int hkv, int r, int h, int block, int split, int part) {
    return ((((size_t)r * hkv + h) * P.blocks + block) * P.splits + split) * (2 * kTileM) + (size_t)part * kTileM;
}

template <bool PREROT, bool LOCAL, bool INTER, bool ALIBI, int PASS>
__global__ void __launch_bounds__(kThreads, 1)
    mass_tc_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap kmap4,
                   const __grid_constant__ CUtensorMap kmap8, const __grid_constant__ CUtensorMap rmap, PoolView pv,
                   MassParams P) {
    constexpr bool ROT = !PREROT && !ALIBI;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ uint64_t bar_kfull[kStages], bar_kempty[kStages], bar_kready[kStages], bar_info[kInfoSlots];
    __shared__ uint64_t bar_sfull[2], bar_sempty[2], bar_qready, bar_drain;
    __shared__ TileInfo s_info[kInfoSlots];
    __shared__ uint32_t s_tmem;
    __shared__ int s_abort;
    __shared__ float2 s_row[PASS == 2 ? 2 * kTileM : 1];   // pass 2: (M, 1 / L) of each row

    // Pass 2's blocks may take an SM as soon as one is free: they build Q before they wait for pass 1's
    // statistics. 2 requests of the 8B shape 39 us for 45 without, 16 requests 102.5 for 101.6, 8 requests of
    // ~17,400 keys 692-704 for 700-722 (timed side by side); the same in pass 2, for the reduction, gains nothing.
    if (PASS == 1) grid_dep_launch_dependents();
    const int pair = blockIdx.x / P.splits, split = blockIdx.x - pair * P.splits;
    const int h = blockIdx.y, r = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = P.g, Hq = pv.hq, Hkv = pv.hkv;
    const int TQ = kTileM / g;
    const int q0 = P.q_offsets[r], q1 = P.q_offsets[r + 1];
    const int i0 = 2 * pair * TQ;
    const int tokens = min(q1 - q0, P.max_rows);
    if (i0 >= tokens) return;
    if (q1 > P.total_q) {
        if (threadIdx.x == 0) record_error(pv.status, LAZYATTN_ERANGE);
        return;
    }
    const int ntok = min(2 * TQ, tokens - i0);
    const bool two = ntok > TQ;                // the second block has rows
    const int m_hi = P.q_start[r] + i0 + ntok - 1;
    const int e0 = P.entry_offsets[r], e1 = min(P.entry_offsets[r + 1], e0 + P.cap);
    const int t_all = e1 > e0 ? (e1 - e0 + kPagesPerTile - 1) / kPagesPerTile : 0;
    const int chunk = (t_all + P.splits - 1) / P.splits;
    const int jb = min(t_all, split * chunk), T = min(t_all, jb + chunk) - jb;

    if (threadIdx.x == 0) {
        s_abort = 0;
        for (int s = 0; s < kStages; ++s) {
            mbar_init(smem_u32(&bar_kfull[s]), 1);
            mbar_init(smem_u32(&bar_kempty[s]), 1);
            mbar_init(smem_u32(&bar_kready[s]), 8);
        }
        for (int s = 0; s < kInfoSlots; ++s) mbar_init(smem_u32(&bar_info[s]), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bar_sfull[i]), 1);
            mbar_init(smem_u32(&bar_sempty[i]), 4);
        }
        mbar_init(smem_u32(&bar_qready), 8);
        mbar_init(smem_u32(&bar_drain), 1);
        mbar_fence_init();
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(&s_tmem), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;
    volatile int* abort_flag = &s_abort;

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        // A K stage is free once the MMAs that read it are done; that also frees the
        // info slot of the tile before: its scores were read before those MMAs were issued.
        // Two sentinels end the stream, one for each warpgroup that takes tiles in turn.
        if (lane == 0) {
            auto load_entries = [&](int jj, uint64_t (&e)[kPagesPerTile], int (&dl)[kPagesPerTile]) {
#pragma unroll
                for (int p = 0; p < kPagesPerTile; ++p) {
                    const int idx = e0 + (jb + jj) * kPagesPerTile + p;
                    const uint64_t v = P.entries[min(idx, e1 - 1)];
                    e[p] = idx < e1 ? v : 0ull;
                    if (LOCAL) dl[p] = P.entry_delta[min(idx, e1 - 1)];
                }
            };
            int last_k[kStages];
#pragma unroll
            for (int s = 0; s < kStages; ++s) last_k[s] = -1;
            uint64_t cur[kPagesPerTile] = {}, nxt[kPagesPerTile] = {};
            int curd[kPagesPerTile] = {}, nxtd[kPagesPerTile] = {};
            if (T > 0) load_entries(0, cur, curd);
            int k = 0;
            bool ok = true;
            for (int j = 0; ok && j < T; ++j) {
                if (j + 1 < T) load_entries(j + 1, nxt, nxtd);
                int n[kPagesPerTile], ys[kPagesPerTile], ss[kPagesPerTile];
                bool live = false, bad = false;
                int consec = 3, full_from = 0;
#pragma unroll
                for (int p = 0; p < kPagesPerTile; ++p) {
                    n[p] = LOCAL ? usable_local(pv, cur[p], curd[p]) : usable_tokens(pv, cur[p]);
                    bad = bad || n[p] < 0;
                    n[p] = max(n[p], 0);
                    ss[p] = entry_start(cur[p]);
                    live = live || (n[p] > 0 && ss[p] <= m_hi);
                    ys[p] = n[p] > 0 ? ((int)entry_page(cur[p]) * Hkv + h) * kPage : P.oob_row;
                    if (n[p] == 0 || entry_page(cur[p]) != entry_page(cur[p & ~3]) + (uint32_t)(p & 3))
                        consec &= ~(1 << (p >> 2));
                    full_from = n[p] == kPage ? max(full_from, ss[p] + kPage - 1) : INT_MAX;
                }
                if (bad) record_error(pv.status, LAZYATTN_ERANGE);
                if (live) {
                    const int st = k % kStages;
                    const int pg0 = (int)entry_page(cur[0]), pg1 = (int)entry_page(cur[4]);
                    if (consec == 3 && pg1 == pg0 + 4) consec |= 4;
                    const int t0 = ss[0];
                    bool strided = ROT && !LOCAL && P.row_blocks > 0 && t0 / kPage + kPagesPerTile <= P.row_blocks;
#pragma unroll
                    for (int p = 0; p < kPagesPerTile; ++p) strided = strided && n[p] > 0 && ss[p] == t0 + kPage * p;
                    ok = k < kStages || mbar_wait(smem_u32(&bar_kempty[st]), ((k / kStages) - 1) & 1, abort_flag);
                    if (!ok) break;
                    const uint32_t fb = smem_u32(&bar_kfull[st]);
                    const uint32_t ds = smem_u32(sm + kOffK + st * 2 * kTile);
                    const uint32_t bs = smem_u32(sm + kOffBase + st * kBaseBytes);
                    mbar_expect_tx(fb, kTile + (ROT ? kBaseBytes : 0));
                    if (consec & 4) {
                        tma_load_4d(ds, &kmap8, 0, 0, h, pg0, fb);
                        tma_load_4d(ds + kHalf, &kmap8, 64, 0, h, pg0, fb);
                    } else {
#pragma unroll
                        for (int b4 = 0; b4 < 2; ++b4) {
                            if (consec & (1 << b4)) {
                                const int pg = b4 ? pg1 : pg0;
                                tma_load_4d(ds + b4 * 8192, &kmap4, 0, 0, h, pg, fb);
                                tma_load_4d(ds + kHalf + b4 * 8192, &kmap4, 64, 0, h, pg, fb);
                            } else {
#pragma unroll
                                for (int p = 4 * b4; p < 4 * b4 + 4; ++p) {
                                    tma_load_2d(ds + p * 2048, &kmap, 0, ys[p], fb);
                                    tma_load_2d(ds + kHalf + p * 2048, &kmap, 64, ys[p], fb);
                                }
                            }
                        }
                    }
                    if (strided) {
                        tma_load_3d(bs, &rmap, 0, t0 % kPage, t0 / kPage, fb);
                    } else if (ROT) {
#pragma unroll
                        for (int p = 0; p < kPagesPerTile; ++p) {
                            const int rowpos = LOCAL ? curd[p] : ss[p];
                            bulk_load(bs + p * 512, pv.rope_pair + (n[p] > 0 ? (size_t)rowpos * (kD / 4) : 0), 512, fb);
                        }
                    }
                    TileInfo& info = s_info[k & (kInfoSlots - 1)];
                    info.j = jb + j;
                    info.full_from = full_from;
#pragma unroll
                    for (int p = 0; p < kPagesPerTile; ++p) {
                        info.start[p] = ss[p];
                        info.n[p] = n[p];
                    }
                    mbar_arrive(smem_u32(&bar_info[k & (kInfoSlots - 1)]));
                    mbar_arrive(fb);
                    last_k[st] = k;
                    ++k;
                }
#pragma unroll
                for (int p = 0; p < kPagesPerTile; ++p) {
                    cur[p] = nxt[p];
                    curd[p] = nxtd[p];
                }
            }
            for (int i = 0; ok && i < 2; ++i, ++k) {
                const int st = k % kStages;
                ok = k < kStages || mbar_wait(smem_u32(&bar_kempty[st]), ((k / kStages) - 1) & 1, abort_flag);
                if (!ok) break;
                s_info[k & (kInfoSlots - 1)].j = -1;
                mbar_arrive(smem_u32(&bar_info[k & (kInfoSlots - 1)]));
                if (i == 0) mbar_arrive(smem_u32(&bar_kfull[st]));
            }
            if (!ok) *abort_flag = 1;
            if (*abort_flag) {   // issued copies land before the CTA's shared memory is released
                volatile int never = 0;
                for (int s = 0; s < kStages; ++s)
                    if (last_k[s] >= 0) mbar_wait(smem_u32(&bar_kfull[s]), (last_k[s] / kStages) & 1, &never);
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        if (lane == 0) {
            const uint32_t id = idesc_f16(kTileM, kN, 0, 0, 0);
            const uint64_t dk = sdesc_sw128(smem_u32(sm + kOffK), 16, 1024);
            // S buffer b gets the scores of row block i
            auto issue = [&](int b, int i, uint64_t ks) {
#pragma unroll
                for (int part = 0; part < 3; ++part) {   // K_lo Q_hi, K_hi Q_lo, K_hi Q_hi
                    const uint64_t ka = ks + (part == 0 ? (uint64_t)(kTile >> 4) : 0);
                    const uint32_t qa = tmem + 256 + i * 128 + (part == 1 ? 64 : 0);
#pragma unroll
                    for (int t = 0; t < kD / 16; ++t)
                        umma_f16_ts(tmem + b * 128, qa + 8 * t, ka + (uint64_t)(((t >> 2) * kHalf + (t & 3) * 32) >> 4), id,
                                    part > 0 || t > 0 ? 1u : 0u);
                }
                umma_commit(smem_u32(&bar_sfull[b]));
            };
            bool ok = mbar_wait(smem_u32(&bar_qready), 0, abort_flag);
            tc_fence_after();
            for (int k = 0; ok; ++k) {
                const int st = k % kStages;
                ok = mbar_wait(smem_u32(&bar_kready[st]), (k / kStages) & 1, abort_flag);
                if (!ok || s_info[k & (kInfoSlots - 1)].j < 0) break;
                const uint64_t ks = dk + (uint64_t)(st * (2 * kTile >> 4));
                if (two) {
                    for (int i = 0; i < 2 && ok; ++i) {
                        ok = k < 1 || mbar_wait(smem_u32(&bar_sempty[i]), (k - 1) & 1, abort_flag);
                        if (!ok) break;
                        tc_fence_after();
                        issue(i, i, ks);
                    }
                    if (!ok) break;
                } else {
                    ok = k < 2 || mbar_wait(smem_u32(&bar_sempty[k & 1]), ((k >> 1) - 1) & 1, abort_flag);
                    if (!ok) break;
                    tc_fence_after();
                    issue(k & 1, 0, ks);
                }
                umma_commit(smem_u32(&bar_kempty[st]));
            }
            umma_commit(smem_u32(&bar_drain));
            volatile int never = 0;
            mbar_wait(smem_u32(&bar_drain), 0, &never);
        }
    } else if (warp >= 12) {
        // ------------------------------------------------------------ K rotation
        // Thread = (page p, half s8 of its slots, frequencies 4u .. 4u + 3). The angle of
        // slot 0 is the page's row of the position table; slot 8's is that plus 8 theta; each
        // next one turns by theta (angle addition, two frequencies an instruction).
        const int rt = threadIdx.x - 384;
        const int p = rt >> 5, s8 = (rt >> 4) & 1, u = rt & 15;
        float2 c1[2], s1[2], ns1[2], c8[2], z8[2];
        if (ROT && !LOCAL) {
            auto row = [&](int pos, int v) {   // the paired table's (cos, cos, sin, sin); positions past it: no key there
                return pos < pv.max_position ? __ldg(pv.rope_pair + (size_t)pos * (kD / 4) + 2 * u + v)
                                             : make_float4(1.f, 1.f, 0.f, 0.f);
            };
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const float4 f = row(1, v), e = row(8 * s8, v);
                c1[v] = make_float2(f.x, f.y);
                s1[v] = make_float2(f.z, f.w);
                ns1[v] = make_float2(-f.z, -f.w);
                c8[v] = make_float2(e.x, e.y);
                z8[v] = make_float2(e.z, e.w);
            }
        }
        auto rot_wait = [&](uint32_t bar, uint32_t parity) {   // one poller; the same answer for all 256 threads
            int go = 1;
            if (rt == 0) go = mbar_wait(bar, parity, abort_flag) ? 1 : 0;
            go = go && *abort_flag == 0;
            int all;
            asm volatile(
                "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.and.pred q, 1, 256, p;\n\t"
                "selp.b32 %0, 1, 0, q;\n\t}"
                : "=r"(all)
                : "r"(go)
                : "memory");
            return all != 0;
        };
        for (int k = 0;; ++k) {
            const int st = k % kStages, ph = (k / kStages) & 1;
            if (!rot_wait(smem_u32(&bar_kfull[st]), ph)) break;
            const TileInfo& info = s_info[k & (kInfoSlots - 1)];
            if (info.j < 0) {
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bar_kready[st]));
                break;
            }
            const int np = info.n[p] - 8 * s8;
            uint8_t* kb = sm + kOffK + st * 2 * kTile + (2 * p + s8) * 1024 + (u & 1) * 8;
            float2 C[2], S[2];
            if (ROT) {
                const float4* b4 = reinterpret_cast<const float4*>(sm + kOffBase + st * kBaseBytes + p * 512) + 2 * u;
#pragma unroll
                for (int v = 0; v < 2; ++v) {
                    const float4 b = b4[v];
                    C[v] = make_float2(b.x, b.y);
                    S[v] = make_float2(b.z, b.w);
                    if (!LOCAL) {
                        const float2 cc = f2_sub(f2_mul(C[v], c8[v]), f2_mul(S[v], z8[v]));
                        S[v] = f2_fma(S[v], c8[v], f2_mul(C[v], z8[v]));
                        C[v] = cc;
                    }
                }
            }
            // two copies: without a test per slot the loads of several slots go out together
            auto rotate = [&](auto WHOLE) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint2* p1 = reinterpret_cast<uint2*>(kb + j * 128 + (((u >> 1) ^ j) << 4));
                uint2* p2 = reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(p1) + kHalf);
                uint2 h1 = make_uint2(0, 0), h2 = h1, l1 = h1, l2 = h1;
                if (WHOLE || j < np) {   // no key in this slot: zeros, so that its scores stay finite
                    const uint2 a = *p1, z = *p2;
                    float2 x[2] = {make_float2(bf_lo(a.x), bf_hi(a.x)), make_float2(bf_lo(a.y), bf_hi(a.y))};
                    float2 y[2] = {make_float2(bf_lo(z.x), bf_hi(z.x)), make_float2(bf_lo(z.y), bf_hi(z.y))};
                    if (ROT) {
#pragma unroll
                        for (int v = 0; v < 2; ++v) {
                            const float2 f = f2_sub(f2_mul(x[v], C[v]), f2_mul(y[v], S[v]));
                            y[v] = f2_fma(x[v], S[v], f2_mul(y[v], C[v]));
                            x[v] = f;
                        }
                    }
                    h1 = make_uint2(pack_h2(x[0].x, x[0].y), pack_h2(x[1].x, x[1].y));
                    h2 = make_uint2(pack_h2(y[0].x, y[0].y), pack_h2(y[1].x, y[1].y));
                    l1 = make_uint2(rest_h2(x[0].x, x[0].y, h1.x), rest_h2(x[1].x, x[1].y, h1.y));
                    l2 = make_uint2(rest_h2(y[0].x, y[0].y, h2.x), rest_h2(y[1].x, y[1].y, h2.y));
                }
                *p1 = h1;
                *p2 = h2;
                *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(p1) + kTile) = l1;
                *reinterpret_cast<uint2*>(reinterpret_cast<uint8_t*>(p2) + kTile) = l2;
                if (ROT && !LOCAL) {   // next slot: angle + theta
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        const float2 cc = f2_fma(C[v], c1[v], f2_mul(S[v], ns1[v]));
                        S[v] = f2_fma(S[v], c1[v], f2_mul(C[v], s1[v]));
                        C[v] = cc;
                    }
                }
            }
            };
            if (np >= 8) rotate(std::true_type{});
            else rotate(std::false_type{});
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&bar_kready[st]));
        }
    } else if (warp >= 4) {
        // ------------------------------------------------------------ rows
        const int wg = (warp - 4) >> 2, quarter = warp & 3;
        const int qi = two ? wg : 0;               // the row block this warpgroup works on
        const int block = 2 * pair + qi;
        const int trow = 32 * quarter + lane;      // row of the block = TMEM lane
        const uint32_t tl = tmem + ((uint32_t)(32 * quarter) << 16);
        const uint32_t ts = tl + wg * 128;         // its S buffer
        const int m0 = P.q_start[r] + block * TQ;  // position of the block's first token
        const int btok = min(TQ, tokens - block * TQ);
        const int t_local = trow / g, jh = trow - t_local * g;
        const int m_row = m0 + t_local;
        bool row_valid = t_local < btok;
        if (row_valid && (m_row < 0 || m_row >= pv.max_position)) {
            record_error(pv.status, LAZYATTN_ERANGE);
            row_valid = false;
        }
        if (two || wg == 0) {   // the row of Q, rotated at m_row and scaled, as hi and lo: dims 2c, 2c + 1 in column c
            const float sc = kLog2e * pv.qk_scale;
            const __nv_bfloat16* qp = P.q + ((size_t)(q0 + block * TQ + t_local) * Hq + (size_t)h * g + jh) * kD;
            const float* cs = reinterpret_cast<const float*>(pv.rope + (size_t)(row_valid ? m_row : 0) * (kD / 2));
            const uint32_t tq = tl + 256 + qi * 128;
#pragma unroll 1
            for (int h4 = 0; h4 < 2; ++h4) {       // 32 dims of each half
                uint32_t hi1[16], hi2[16], lo1[16], lo2[16];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int u = 4 * h4 + i;
                    uint4 a1 = make_uint4(0, 0, 0, 0), a2 = a1, b1 = a1, b2 = a1;
                    if (row_valid) {
                        uint4 a = __ldg(reinterpret_cast<const uint4*>(qp + (INTER ? 16 * u : 8 * u)));
                        uint4 b = __ldg(reinterpret_cast<const uint4*>(qp + (INTER ? 16 * u + 8 : 64 + 8 * u)));
                        if (INTER) deinterleave16(a, b, a, b);
                        float x1[8], x2[8], n2 = 0.f;
                        unpack8(a, x1);
                        unpack8(b, x2);
#pragma unroll
                        for (int v = 0; v < 8; ++v) n2 = fmaxf(n2, fmaf(x1[v], x1[v], x2[v] * x2[v]));
                        if (!(n2 * sc * sc <= kMaxPairNorm2)) record_error(pv.status, LAZYATTN_ERANGE);
                        const float4* c4 = reinterpret_cast<const float4*>(cs + 16 * u);
#pragma unroll
                        for (int v = 0; v < 4; ++v) {
                            const float4 f = ALIBI ? make_float4(1.f, 0.f, 1.f, 0.f) : __ldg(c4 + v);
                            const float a0 = x1[2 * v], z0 = x2[2 * v], a1_ = x1[2 * v + 1], z1 = x2[2 * v + 1];
                            x1[2 * v] = (a0 * f.x - z0 * f.y) * sc;
                            x2[2 * v] = (a0 * f.y + z0 * f.x) * sc;
                            x1[2 * v + 1] = (a1_ * f.z - z1 * f.w) * sc;
                            x2[2 * v + 1] = (a1_ * f.w + z1 * f.z) * sc;
                        }
                        split8(x1, a1, b1);
                        split8(x2, a2, b2);
                    }
                    hi1[4 * i] = a1.x; hi1[4 * i + 1] = a1.y; hi1[4 * i + 2] = a1.z; hi1[4 * i + 3] = a1.w;
                    hi2[4 * i] = a2.x; hi2[4 * i + 1] = a2.y; hi2[4 * i + 2] = a2.z; hi2[4 * i + 3] = a2.w;
                    lo1[4 * i] = b1.x; lo1[4 * i + 1] = b1.y; lo1[4 * i + 2] = b1.z; lo1[4 * i + 3] = b1.w;
                    lo2[4 * i] = b2.x; lo2[4 * i + 1] = b2.y; lo2[4 * i + 2] = b2.z; lo2[4 * i + 3] = b2.w;
                }
                __syncwarp();
                tmem_st16(tq + 16 * h4, hi1);
                tmem_st16(tq + 32 + 16 * h4, hi2);
                tmem_st16(tq + 64 + 16 * h4, lo1);
                tmem_st16(tq + 96 + 16 * h4, lo2);
            }
            tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&bar_qready));

        // pass 2: this thread's four rows in the fragment layout: 32 quarter + lane / 4 + 8 f
        float nM[4], inv[4], slope4[4];
        int m4[4];
        int m_see = INT_MAX;   // smallest position of the warp's rows with weights
        if (PASS == 2) {
            grid_dep_wait();
            {   // merge the row's statistics
                float M = -INFINITY, Lsum = 0.f;
                for (int i = 0; i < 2 * P.splits; ++i) {
                    const float2 x = P.stats[stats_at(P, Hkv, r, h, block, i >> 1, i & 1) + trow];
                    if (x.y > 0.f) M = fmaxf(M, x.x);
                }
                for (int i = 0; i < 2 * P.splits && M != -INFINITY; ++i) {
                    const float2 x = P.stats[stats_at(P, Hkv, r, h, block, i >> 1, i & 1) + trow];
                    if (x.y > 0.f) Lsum += x.y * fast_exp2(x.x - M);
                }
                s_row[wg * kTileM + trow] = Lsum > 0.f ? make_float2(M, 1.f / Lsum) : make_float2(0.f, 0.f);
            }
            __syncwarp();      // a warp reads the rows of its own lanes only
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                const int row = 32 * quarter + (lane >> 2) + 8 * f;
                const float2 x = s_row[wg * kTileM + row];
                nM[f] = x.y > 0.f ? -x.x : -INFINITY;   // a row that sees no key: weights 0 whatever its scores
                inv[f] = x.y;
                m4[f] = m0 + row / g;
                slope4[f] = ALIBI ? alibi_slope(h * g + row % g, Hq) * kLog2e : 0.f;
                if (x.y > 0.f) m_see = min(m_see, m4[f]);
            }
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) m_see = min(m_see, __shfl_xor_sync(0xffffffffu, m_see, o));
        }

        float m_run = -INFINITY, l_run = 0.f;
        bool ok = true;
        const float slope = ALIBI ? alibi_slope(h * g + jh, Hq) * kLog2e : 0.f;
        for (int k = two ? 0 : wg, use = 0;; k += two ? 1 : 2, ++use) {
            const int is = k & (kInfoSlots - 1);
            ok = mbar_wait(smem_u32(&bar_info[is]), (k / kInfoSlots) & 1, abort_flag);
            const TileInfo& info = s_info[is];
            const int j = ok ? info.j : -1;
            // The S buffer is free once its last columns are in registers: the next MMAs overlap
            // the arithmetic on those. (The tile info stays: its slot is reused 8 tiles on.)
            auto release = [&] {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&bar_sempty[wg]));
            };
            if (PASS == 1) {
                if (j < 0) break;
                // (rows without a query count as seeing all: their sums are dropped at the end)
                const bool wfull = __all_sync(0xffffffffu, row_valid ? m_row >= info.full_from : info.full_from != INT_MAX);
                ok = mbar_wait(smem_u32(&bar_sfull[wg]), use & 1, abort_flag);
                if (!ok) break;
                tc_fence_after();
#pragma unroll 1   // (unrolled, a pass of few tiles spends its time fetching instructions)
                for (int w = 0; w < 4; ++w) {   // pages 2w and 2w + 1
                    uint32_t v[32];
                    tmem_ld32(ts + 32 * w, v);
                    if (w == 3) release();
                    if (ALIBI) {
                        const int d0 = info.start[2 * w] - m_row, d1 = info.start[2 * w + 1] - m_row;
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            v[i] = __float_as_uint(__uint_as_float(v[i]) + slope * (float)((i < 16 ? d0 : d1) + (i & 15)));
                    }
                    if (!wfull) {
                        uint32_t vis = 0;   // bit i: the row sees the key of column i
#pragma unroll
                        for (int hp = 0; hp < 2; ++hp) {
                            const int p = 2 * w + hp;
                            const int l = row_valid ? max(min(info.n[p], m_row - info.start[p] + 1), 0) : 0;
                            vis |= ((1u << l) - 1u) << (16 * hp);
                        }
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = (vis >> i) & 1u ? v[i] : 0xff800000u;
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        mx[i & 3] = fmax3(mx[i & 3], __uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
                    if (top > m_run + kRescaleThreshold) {
                        l_run *= fast_exp2(m_run - top);   // 0 while m_run is -inf
                        m_run = top;
                    }
                    const float ref = m_run == -INFINITY ? 0.f : m_run;
                    float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 d = f2_sub(make_float2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])),
                                                make_float2(ref, ref));
                        sum[i & 1] = f2_add(sum[i & 1], make_float2(fast_exp2(d.x), fast_exp2(d.y)));
                    }
                    const float2 both = f2_add(sum[0], sum[1]);
                    l_run += both.x + both.y;
                }
            } else {
                const bool full = j >= 0 && info.full_from <= m_see;   // every key is seen by every row with weights
                float* cols = reinterpret_cast<float*>(sm + kOffSum) + ((wg * 2 + (use & 1)) * 4 + quarter) * kN;
                ok = j >= 0 && mbar_wait(smem_u32(&bar_sfull[wg]), use & 1, abort_flag);
                tc_fence_after();
                // two copies of the work, so that a tile without a hidden key tests nothing
                auto weights = [&](auto FULL) {
#pragma unroll 1
                for (int w = 0; w < 4; ++w) {
                    uint32_t v[2][16];
                    tmem_ld_frag32(ts + 32 * w, v[0]);
                    tmem_ld_frag32(ts + 32 * w + (16u << 16), v[1]);
                    if (w == 3) release();
                    float2 acc[4];   // columns 32 w + 8 i + 2 (lane % 4), + 1
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[i] = make_float2(0.f, 0.f);
                        const int p = 2 * w + (i >> 1), s0 = 8 * (i & 1) + 2 * (lane & 3);
                        const int pos = (ALIBI || !FULL) ? info.start[p] + s0 : 0;
                        const int n = FULL ? kPage : info.n[p];
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            float2 d = make_float2(__uint_as_float(v[f >> 1][4 * i + 2 * (f & 1)]),
                                                   __uint_as_float(v[f >> 1][4 * i + 2 * (f & 1) + 1]));
                            if (ALIBI) {
                                d.x += slope4[f] * (float)(pos - m4[f]);
                                d.y += slope4[f] * (float)(pos + 1 - m4[f]);
                            }
                            d = f2_add(d, make_float2(nM[f], nM[f]));
                            if (!FULL) {
                                d.x = s0 < n && pos <= m4[f] ? d.x : -INFINITY;
                                d.y = s0 + 1 < n && pos + 1 <= m4[f] ? d.y : -INFINITY;
                            }
                            acc[i] = f2_fma(make_float2(fast_exp2(d.x), fast_exp2(d.y)), make_float2(inv[f], inv[f]), acc[i]);
                        }
                    }
                    // join the 8 threads of a column (lane / 4), halving the columns each time
                    float a4[4], a2[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {   // lane bit 4 picks column groups 2, 3
                        const bool up = lane & 16;
                        const float2 give = up ? acc[i] : acc[i + 2], keep = up ? acc[i + 2] : acc[i];
                        a4[2 * i] = keep.x + __shfl_xor_sync(0xffffffffu, give.x, 16);
                        a4[2 * i + 1] = keep.y + __shfl_xor_sync(0xffffffffu, give.y, 16);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {   // lane bit 3: the second group of the two
                        const bool up = lane & 8;
                        a2[i] = (up ? a4[2 + i] : a4[i]) + __shfl_xor_sync(0xffffffffu, up ? a4[i] : a4[2 + i], 8);
                    }
                    const bool up = lane & 4;       // lane bit 2: the second column of the pair
                    const float a1 = (up ? a2[1] : a2[0]) + __shfl_xor_sync(0xffffffffu, up ? a2[0] : a2[1], 4);
                    cols[32 * w + ((lane >> 4) & 1) * 16 + ((lane >> 3) & 1) * 8 + 2 * (lane & 3) + ((lane >> 2) & 1)] = a1;
                }
                };
                if (ok) {
                    if (full) weights(std::true_type{});
                    else weights(std::false_type{});
                }
                const int idx = j * kPagesPerTile + (trow >> 4);
                // The four warps meet (the other parity's buffer is free: all have passed the last
                // meeting). A warp that gave up or saw the last tile says so here and all leave
                // together: none is left waiting.
                int all_ok;
                asm volatile(
                    "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.and.pred q, %2, 128, p;\n\t"
                    "selp.b32 %0, 1, 0, q;\n\t}"
                    : "=r"(all_ok)
                    : "r"(ok ? 1 : 0), "r"(2 + wg)
                    : "memory");
                if (!all_ok) break;
                const float* all = reinterpret_cast<const float*>(sm + kOffSum) + (wg * 2 + (use & 1)) * 4 * kN + trow;
                if (idx < e1 - e0)
                    P.sums[((((size_t)block * P.requests + r) * P.cap + idx) * Hkv + h) * kPage + (trow & 15)] =
                        (all[0] + all[kN]) + (all[2 * kN] + all[3 * kN]);
            }
        }
        if (PASS == 1) {
            // two blocks: each has one part, the other stays empty; one block: a part from each warpgroup
            const float2 x = make_float2(m_run == -INFINITY ? 0.f : m_run, ok && row_valid ? l_run : 0.f);
            P.stats[stats_at(P, Hkv, r, h, block, split, two ? 0 : wg) + trow] = x;
            if (two) P.stats[stats_at(P, Hkv, r, h, block, split, 1) + trow] = make_float2(0.f, 0.f);
        }
    }

    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && s_abort) record_error(pv.status, LAZYATTN_EDEVICE);
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
}

// Thread = (entry, KV head, slot): the row blocks' sums in order. A block has written an
// entry's sums iff the entry starts at or before the block's last row.
template <bool LOCAL>
__global__ void __launch_bounds__(256)
    mass_reduce_kernel(PoolView pv, MassParams P, const float* mass_in, float* mass_out, float decay) {
    const int r = blockIdx.y;
    const int per = pv.hkv * kPage;
    grid_dep_wait();
    const int e0 = P.entry_offsets[r], E = P.entry_offsets[r + 1] - e0;
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int i = (int)(at / per), rest = (int)(at - (int64_t)i * per);
    if (at == 0 && E > P.cap) record_error(pv.status, LAZYATTN_ERANGE);
    if (i >= min(E, P.cap)) return;
    const uint64_t e = P.entries[e0 + i];
    const int n = LOCAL ? usable_local(pv, e, P.entry_delta[e0 + i]) : usable_tokens(pv, e);
    const size_t to = (size_t)(e0 + i) * per + rest;
    float sum = 0.f;
    if ((rest & 15) < n) {
        const int q0 = P.q_offsets[r], q1 = P.q_offsets[r + 1];
        const int tokens = q1 <= P.total_q ? min(q1 - q0, P.max_rows) : 0;
        const int TQ = kTileM / P.g, m0 = P.q_start[r];
        for (int b = 0; b * TQ < tokens; ++b)
            if (entry_start(e) <= m0 + min((b + 1) * TQ, tokens) - 1)
                sum += P.sums[(((size_t)b * P.requests + r) * P.cap + i) * per + rest];
        if (mass_in) sum += decay * mass_in[to];
    }
    mass_out[to] = sum;
}

using MassKernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const CUtensorMap, PoolView,
                            MassParams);

template <int PASS>
MassKernel mass_kernel_for(bool prerot, bool local, bool inter, bool alibi) {
    if (alibi) return mass_tc_kernel<false, false, false, true, PASS>;
    if (local) return inter ? mass_tc_kernel<false, true, true, false, PASS> : mass_tc_kernel<false, true, false, false, PASS>;
    if (prerot) return inter ? mass_tc_kernel<true, false, true, false, PASS> : mass_tc_kernel<true, false, false, false, PASS>;
    return inter ? mass_tc_kernel<false, false, true, false, PASS> : mass_tc_kernel<false, false, false, false, PASS>;
}

inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

struct MassWs {
    int blocks, splits;
    size_t sums_off, total;
};

// CTAs per (request, KV head, two row blocks): the split with the least time by waves of
// CTAs, each its tiles plus a start and an end of about four tiles' time; shares of 4 tiles or more.
MassWs mass_ws(const lazyattn_pool& p, const lazyattn_batch& b) {
    MassWs w;
    const int g = p.d.n_q_heads / p.d.n_kv_heads, TQ = kTileM / g;
    w.blocks = 2 * std::max(1, (b.max_q_len + 2 * TQ - 1) / (2 * TQ));
    const int64_t items = (int64_t)b.num_requests * p.d.n_kv_heads * (w.blocks / 2);
    const int64_t T = ((int64_t)b.max_entries + kPagesPerTile - 1) / kPagesPerTile;
    const int64_t sms = p.sm_count > 0 ? p.sm_count : 1;
    w.splits = 1;
    double best = 0.0;
    for (int s = 1; s <= 16; ++s) {
        if (s > 1 && T / s < 4) break;
        const double cost = (double)((items * s + sms - 1) / sms) * ((double)((T + s - 1) / s) + 4.0);
        if (s == 1 || cost < best) {
            best = cost;
            w.splits = s;
        }
    }
    w.sums_off = up256((size_t)items * 2 * w.splits * 2 * kTileM * sizeof(float2));
    w.total = w.sums_off + up256((size_t)w.blocks * b.num_requests * (size_t)std::max(b.max_entries, 1) *
                                 p.d.n_kv_heads * kPage * sizeof(float));
    return w;
}

}  // namespace

int mass_tc_init() {
    for (int i = 0; i < 9; ++i) {
        if (i < 8 && (i & 1) && (i & 2)) continue;   // pre-rotated pages are never doc-local
        const bool alibi = i == 8;
        MassKernel k1 = mass_kernel_for<1>(!alibi && (i & 1), !alibi && (i & 2), !alibi && (i & 4), alibi);
        MassKernel k2 = mass_kernel_for<2>(!alibi && (i & 1), !alibi && (i & 2), !alibi && (i & 4), alibi);
        if (cudaFuncSetAttribute(k1, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess ||
            cudaFuncSetAttribute(k2, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess)
            return LAZYATTN_ECUDA;
    }
    return LAZYATTN_OK;
}

size_t mass_tc_ws_bytes(const lazyattn_pool& p, const lazyattn_batch& b) { return mass_ws(p, b).total; }

int launch_prefill_mass_bf16(const lazyattn_pool& p, const lazyattn_batch& b, const __nv_bfloat16* q,
                             const float* mass_in, float* mass_out, float decay, void* ws, cudaStream_t stream) {
    if (!p.have_maps) return LAZYATTN_ECUDA;
    if (b.max_entries < 1) return LAZYATTN_OK;
    const MassWs w = mass_ws(p, b);
    MassParams P;
    P.entries = b.entries;
    P.entry_offsets = b.entry_offsets;
    P.entry_delta = b.entry_delta;
    P.q_offsets = b.q_offsets;
    P.q_start = b.q_start;
    P.q = q;
    P.total_q = b.total_q;
    P.max_rows = b.max_q_len;
    P.g = p.d.n_q_heads / p.d.n_kv_heads;
    P.oob_row = (int32_t)((uint64_t)p.d.num_pages * (uint64_t)p.d.n_kv_heads * kPage);
    P.row_blocks = p.have_rmap ? p.d.max_position / kPage : 0;
    P.blocks = w.blocks;
    P.splits = w.splits;
    P.cap = b.max_entries;
    P.requests = b.num_requests;
    P.stats = static_cast<float2*>(ws);
    P.sums = reinterpret_cast<float*>(static_cast<char*>(ws) + w.sums_off);
    const bool prerot = (b.flags & LAZYATTN_KEYS_PREROTATED) != 0, inter = p.d.rope_interleaved != 0;
    const bool local = p.d.key_storage == LAZYATTN_KEYS_DOC_LOCAL, alibi = p.d.position_encoding == LAZYATTN_POS_ALIBI;
    if (b.total_q > 0 && b.max_q_len > 0) {
        const dim3 grid(w.blocks / 2 * w.splits, p.d.n_kv_heads, b.num_requests);
        mass_kernel_for<1>(prerot, local, inter, alibi)<<<grid, kThreads, kSmemBytes, stream>>>(p.kmap, p.kmap4, p.kmap8,
                                                                                                p.rmap, p.view(), P);
        if (cudaGetLastError() != cudaSuccess ||
            launch_dependent(mass_kernel_for<2>(prerot, local, inter, alibi), grid, dim3(kThreads), kSmemBytes, stream,
                             p.kmap, p.kmap4, p.kmap8, p.rmap, p.view(), P) != cudaSuccess)
            return LAZYATTN_ECUDA;
    } else {
        P.max_rows = 0;
    }
    const int64_t threads = (int64_t)b.max_entries * p.d.n_kv_heads * kPage;
    if (launch_dependent(local ? mass_reduce_kernel<true> : mass_reduce_kernel<false>,
                         dim3((unsigned)((threads + 255) / 256), b.num_requests), dim3(256), 0, stream, p.view(), P, mass_in,
                         mass_out, decay) != cudaSuccess)
        return LAZYATTN_ECUDA;
    return cudaGetLastError() == cudaSuccess ? LAZYATTN_OK : LAZYATTN_ECUDA;
}

}  // namespace lazyattn
