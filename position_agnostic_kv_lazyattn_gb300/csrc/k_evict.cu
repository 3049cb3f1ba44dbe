// Eviction by accumulated attention weight: per (request, KV head), choose the
// tokens to keep and copy their K and V into the request's new pages.
//
// One block per (KV head, request). Tokens are numbered in table order. The
// k-th largest mass among the tokens that are neither sinks nor recent is found by
// a radix select, most significant byte first, over the masses as ordered
// integers; of the tokens equal to it the earliest are taken. The kept tokens'
// places go to `kept` in order, then each is replaced by the token's position as
// its rows are copied.
#include "internal.h"

namespace lazyattn {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// Order-preserving integer of a mass (larger mass, larger integer): NaN is 0, the
// least; -0 and 0 are equal.
__device__ __forceinline__ uint32_t mass_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sums of a block's (a, b) pairs, and the totals. Called by all threads.
__device__ __forceinline__ int2 block_scan(int2 v, int2 (&warp_sum)[kWarps], int2& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int2 x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, x.x, o), b = __shfl_up_sync(0xffffffffu, x.y, o);
        if (lane >= o) {
            x.x += a;
            x.y += b;
        }
    }
    __syncthreads();   // the sums of an earlier call have been read
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int2 before = make_int2(0, 0);
    total = make_int2(0, 0);
    for (int w = 0; w < kWarps; ++w) {
        if (w == warp) before = total;
        total.x += warp_sum[w].x;
        total.y += warp_sum[w].y;
    }
    return make_int2(before.x + x.x - v.x, before.y + x.y - v.y);
}

struct EvictParams {
    const uint64_t* entries;
    const int32_t* entry_offsets;
    const float* mass;
    uint64_t* dst_entries;
    const int32_t* dst_offsets;
    int32_t* kept;
    float* dst_mass;
    int32_t budget, sinks, recent;
    int32_t row_vecs;   // 16-byte vectors of a K or V row
};

__global__ void __launch_bounds__(kThreads) evict_kernel(PoolView pv, EvictParams P) {
    const int h = blockIdx.x, r = blockIdx.y, tid = threadIdx.x;
    const int hkv = pv.hkv;
    const int e0 = P.entry_offsets[r], E = P.entry_offsets[r + 1] - e0;
    const int d0 = P.dst_offsets[r], DE = P.dst_offsets[r + 1] - d0;
    int32_t* kept = P.kept + ((size_t)r * hkv + h) * P.budget;
    __shared__ int2 s_sum[kWarps];
    __shared__ int s_hist[256];
    __shared__ int s_bad;
    __shared__ uint32_t s_key;
    __shared__ int s_need;
    if (tid == 0) s_bad = 0;
    __syncthreads();

    // Count the tokens and check the table: pages and positions in range, entries with tokens
    // ascending in position (each against the last one before it that has tokens).
    int n_tok = 0;
    for (int base = 0; base < E; base += kThreads) {
        const int i = base + tid;
        const uint64_t e = i < E ? P.entries[e0 + i] : 0ull;
        const int n = entry_nvalid(e);
        if (n > 0 && !entry_ok(pv, e)) s_bad = 1;
        if (n > 0) {
            for (int k = i - 1; k >= 0; --k) {
                const uint64_t f = P.entries[e0 + k];
                if (entry_nvalid(f) == 0) continue;
                if (entry_start(f) + entry_nvalid(f) > entry_start(e)) s_bad = 1;
                break;
            }
        }
        int2 total;
        block_scan(make_int2(min(n, kPage), 0), s_sum, total);
        n_tok += total.x;
    }
    const int count = min(n_tok, P.budget);
    const int pages = (count + kPage - 1) / kPage;
    if (tid == 0 && (DE < pages || DE > (LAZYATTN_MAX_START + 1) / kPage)) s_bad = 1;
    for (int i = tid; i < min(DE, pages); i += kThreads)
        if ((uint32_t)P.dst_entries[d0 + i] >= (uint32_t)pv.num_pages) s_bad = 1;
    __syncthreads();
    const bool bad = s_bad != 0;
    if (bad && tid == 0) record_error(pv.status, LAZYATTN_ERANGE);
    const int cnt = bad ? 0 : count;

    // New entries: the upper word holds start, count and the writable bit.
    if (h == 0)
        for (int i = tid; i < DE; i += kThreads) {
            uint32_t* hi = reinterpret_cast<uint32_t*>(P.dst_entries + d0 + i) + 1;
            const uint32_t start = (uint32_t)min((int64_t)i * kPage, (int64_t)LAZYATTN_MAX_START);
            *hi = (*hi & 0x80000000u) | start | ((uint32_t)max(0, min(kPage, cnt - i * kPage)) << 26);
        }

    auto mass_at = [&](int i, int s) { return P.mass[((size_t)(e0 + i) * hkv + h) * kPage + s]; };
    const int lo = min(P.sinks, n_tok), hi = max(lo, n_tok - P.recent);   // tokens [lo, hi) compete
    const int need = cnt - (n_tok - (hi - lo));                          // of them this many stay
    const bool all = cnt == n_tok;
    uint32_t key = 0;       // the smallest kept mass
    int equal = 0;          // how many tokens equal to it stay
    if (!bad && !all) {
        int want = need;
        for (int shift = 24; shift >= 0; shift -= 8) {
            for (int b = tid; b < 256; b += kThreads) s_hist[b] = 0;
            __syncthreads();
            int at = 0;
            for (int base = 0; base < E; base += kThreads) {
                const int i = base + tid;
                const int n = i < E ? entry_nvalid(P.entries[e0 + i]) : 0;
                int2 total;
                const int first = at + block_scan(make_int2(n, 0), s_sum, total).x;
                at += total.x;
                for (int s = 0; s < n; ++s) {
                    const int t = first + s;
                    if (t < lo || t >= hi) continue;
                    const uint32_t k = mass_key(mass_at(i, s));
                    if (shift == 24 || (k >> (shift + 8)) == (key >> (shift + 8))) atomicAdd(&s_hist[(k >> shift) & 255], 1);
                }
            }
            __syncthreads();
            if (tid == 0) {
                int above = 0, b = 255;
                for (; b > 0 && above + s_hist[b] < want; --b) above += s_hist[b];
                s_key = key | ((uint32_t)b << shift);
                s_need = want - above;
            }
            __syncthreads();
            key = s_key;
            want = s_need;
        }
        equal = want;
    }

    // Places of the kept tokens, in table order.
    if (!bad) {
        int at = 0, at_eq = 0, at_kept = 0;
        for (int base = 0; base < E; base += kThreads) {
            const int i = base + tid;
            const int n = i < E ? entry_nvalid(P.entries[e0 + i]) : 0;
            int2 total;
            const int first = at + block_scan(make_int2(n, 0), s_sum, total).x;
            at += total.x;
            uint32_t gt = 0, eq = 0;   // slots kept for sure; slots equal to the threshold
            for (int s = 0; s < n; ++s) {
                const int t = first + s;
                if (all || t < lo || t >= hi) {
                    gt |= 1u << s;
                } else {
                    const uint32_t k = mass_key(mass_at(i, s));
                    if (k > key) gt |= 1u << s;
                    if (k == key) eq |= 1u << s;
                }
            }
            const int eq_before = at_eq + block_scan(make_int2(__popc(eq), 0), s_sum, total).x;
            at_eq += total.x;
            int take = max(0, min(__popc(eq), equal - eq_before));
            for (uint32_t todo = eq; take > 0; todo &= todo - 1, --take) gt |= todo & -todo;
            int to = at_kept + block_scan(make_int2(__popc(gt), 0), s_sum, total).x;
            at_kept += total.x;
            for (uint32_t todo = gt; todo; todo &= todo - 1, ++to) kept[to] = i * kPage + __ffs(todo) - 1;
        }
    }
    __syncthreads();

    // Copy: `vecs` threads per token; slots of the last page past the tokens become zeros.
    const int vecs = P.row_vecs, per = kThreads / vecs, v = tid % vecs;
    uint4* kp = static_cast<uint4*>(pv.k_pool);
    uint4* vp = static_cast<uint4*>(pv.v_pool);
    const int used = (cnt + kPage - 1) / kPage * kPage;
    for (int j = tid / vecs; j < used; j += per) {
        const uint32_t page = (uint32_t)P.dst_entries[d0 + j / kPage];
        const size_t dst = (((size_t)page * hkv + h) * kPage + j % kPage) * vecs + v;
        uint4 a = make_uint4(0, 0, 0, 0), b = a;
        if (j < cnt) {
            const int code = kept[j];
            const uint64_t e = P.entries[e0 + code / kPage];
            const size_t src = (((size_t)entry_page(e) * hkv + h) * kPage + code % kPage) * vecs + v;
            a = kp[src];
            b = vp[src];
            if (v == 0 && P.dst_mass)
                P.dst_mass[((size_t)(d0 + j / kPage) * hkv + h) * kPage + j % kPage] = mass_at(code / kPage, code % kPage);
        } else if (v == 0 && P.dst_mass) {
            P.dst_mass[((size_t)(d0 + j / kPage) * hkv + h) * kPage + j % kPage] = 0.f;
        }
        kp[dst] = a;
        vp[dst] = b;
    }
    __syncthreads();
    for (int j = tid; j < P.budget; j += kThreads)
        kept[j] = j < cnt ? entry_start(P.entries[e0 + kept[j] / kPage]) + kept[j] % kPage : -1;
    if (P.dst_mass)
        for (int j = used + tid; j < DE * kPage; j += kThreads)
            P.dst_mass[((size_t)(d0 + j / kPage) * hkv + h) * kPage + j % kPage] = 0.f;
}

}  // namespace

int launch_evict(const lazyattn_pool& p, const lazyattn_batch& b, const float* mass, int32_t budget, int32_t sinks,
                 int32_t recent, uint64_t* dst_entries, const int32_t* dst_offsets, int32_t* kept, float* dst_mass,
                 cudaStream_t stream) {
    EvictParams P;
    P.entries = b.entries;
    P.entry_offsets = b.entry_offsets;
    P.mass = mass;
    P.dst_entries = dst_entries;
    P.dst_offsets = dst_offsets;
    P.kept = kept;
    P.dst_mass = dst_mass;
    P.budget = budget;
    P.sinks = sinks;
    P.recent = recent;
    P.row_vecs = p.d.head_dim * (p.d.dtype == LAZYATTN_F32 ? 4 : 2) / 16;
    evict_kernel<<<dim3(p.d.n_kv_heads, b.num_requests), kThreads, 0, stream>>>(p.view(), P);
    return cudaGetLastError() == cudaSuccess ? LAZYATTN_OK : LAZYATTN_ECUDA;
}

}  // namespace lazyattn
