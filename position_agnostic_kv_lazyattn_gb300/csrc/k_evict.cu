// Eviction by accumulated attention weight: per (request, KV head), choose the
// tokens to keep and copy their K and V into the request's new pages.
//
// One cluster of 1..8 blocks per (KV head, request); each block has a contiguous
// share of the table's entries. Tokens are numbered in table order. The k-th
// largest mass among the tokens that are neither sinks nor recent is found by a radix
// select over the masses as ordered integers, 11 bits at a time: every block counts its share
// into a histogram in shared memory, and every block reads all the cluster's
// histograms and finds the digit for itself, so a digit takes one cluster barrier. Of
// the tokens equal to the threshold the earliest are taken. The kept tokens' places go
// to `kept` in order. No order of execution shows in the result: counts are integers,
// places come from prefix sums. A second kernel copies the rows, which is all of
// the memory traffic that counts, over the whole GPU (in the selecting blocks, each wave's
// copies waited for its selection: 32 requests cut to 2048 tokens took 156 us).
//
// The masses are read from memory once (a share of up to 2048 entries stays in shared memory as
// integers; larger ones are read again for every digit).
//
// Measured (GB300): 32 requests of ~9,200 tokens cut to 2048, 8 heads: 115-116 us, the
// selection 26 (latency of its phases) and the copy 86 (537 MB at 6.2 TB/s: bound by memory); one request
// of 2,118 tokens cut to 512: 14.5 us in a graph, 16-18 from Python.
#include <cooperative_groups.h>
#include <limits.h>

#include "internal.h"

namespace cg = cooperative_groups;

namespace lazyattn {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kSeg = 2048;                  // entries of a share held in shared memory at a time
constexpr int kRun = kSeg / kThreads;       // consecutive entries a thread scans
constexpr int kBits = 11, kBins = 1 << kBits;
constexpr int kDigits = 3;                  // bits 21..31, 10..20, 0..9
constexpr int kMaxCluster = 8;
constexpr uint32_t kKeep = 0xffffffffu;     // key of a sink or a recent token
constexpr uint32_t kNone = 0xfffffffeu;     // key of a slot without a token (masses end at 0xff800000)

// Order-preserving integer of a mass (larger mass, larger integer): NaN is 0, the
// least; -0 and 0 are equal.
__device__ __forceinline__ uint32_t mass_key(float x) {
    if (x != x) return 0u;
    const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Exclusive sum over the block, and the total. Called by all threads.
__device__ __forceinline__ int block_scan(int v, int (&warp_sum)[kWarps], int& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += a;
    }
    __syncthreads();   // the sums of an earlier call have been read
    if (lane == 31) warp_sum[warp] = x;
    __syncthreads();
    int before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    return before + x - v;
}

// Largest value of the threads before this one (0 for the first; values are 0 or more), and of all.
__device__ __forceinline__ int block_max_before(int v, int (&warp_max)[kWarps], int& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int a = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x = max(x, a);
    }
    __syncthreads();   // the values of an earlier call have been read
    if (lane == 31) warp_max[warp] = x;
    __syncthreads();
    int before = 0;
    all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) before = max(before, warp_max[w]);
        all = max(all, warp_max[w]);
    }
    const int up = __shfl_up_sync(0xffffffffu, x, 1);
    return lane ? max(before, up) : before;
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
    int32_t cap;         // entries per request (host bound, by which the copy is sized)
    int32_t seg;         // entries of a share held at a time (at most kSeg)
};

struct Shared {
    int hist[kDigits][kBins];
    int scan[kWarps];
    int tokens, bad;           // of this block's share
    int first, end;            // its first token's position (INT_MAX: none), the largest position + 1 of its tokens
    int sure, equal;           // tokens kept for certain, tokens equal to the threshold
    int digit, want;
    int warp_sure[kWarps], warp_equal[kWarps];
};

__global__ void __launch_bounds__(kThreads, 2) evict_kernel(PoolView pv, EvictParams P) {
    extern __shared__ __align__(16) uint32_t dyn[];
    __shared__ Shared S;
    cg::cluster_group cluster = cg::this_cluster();
    // The copy's blocks wait for this grid's end before they read anything it writes: 13.7 us for 14.0 a small
    // call in a graph, 115 for 116 with 32 requests.
    grid_dep_launch_dependents();
    const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int h = blockIdx.y, r = blockIdx.z, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int hkv = pv.hkv;
    const int e0 = P.entry_offsets[r], E = P.entry_offsets[r + 1] - e0;
    const int d0 = P.dst_offsets[r], DE = P.dst_offsets[r + 1] - d0;
    int32_t* kept = P.kept + ((size_t)r * hkv + h) * P.budget;
    const int per = (E + C - 1) / C;
    const int a0 = min(E, rank * per), a1 = min(E, a0 + per);   // this block's entries
    const int segs = (a1 - a0 + P.seg - 1) / P.seg;
    uint32_t* keys = dyn;                                        // [seg][16]
    int* first = reinterpret_cast<int*>(dyn + (size_t)P.seg * kPage);   // [seg]: tokens before the entry, in the share

    for (int b = tid; b < kDigits * kBins; b += kThreads) (&S.hist[0][0])[b] = 0;
    if (tid == 0) {
        S.bad = 0;
        S.first = INT_MAX;
        S.end = 0;
    }
    __syncthreads();

    // Count the share's tokens and check the table: pages and positions in range, entries
    // with tokens ascending in position (each starts at or past the ends of all before it).
    // Leaves the segment's `first`, and the tokens before the segment in `before`.
    auto load_entries = [&](int seg, int before, bool check) {
        const int b0 = a0 + seg * P.seg, n_here = min(P.seg, a1 - b0);
        int n[kRun], sum = 0, begin[kRun], end = 0;
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            const int i = tid * kRun + j;
            const uint64_t e = i < n_here ? P.entries[e0 + b0 + i] : 0ull;
            n[j] = min(entry_nvalid(e), kPage);
            sum += n[j];
            begin[j] = entry_start(e);
            if (check && n[j] > 0) {
                if (!entry_ok(pv, e)) S.bad = 1;
                end = max(end, begin[j] + n[j]);
            }
        }
        if (check) {
            int all;
            int so_far = max(block_max_before(end, S.scan, all), S.end);   // S.end: of the segments before
#pragma unroll
            for (int j = 0; j < kRun; ++j) {
                if (n[j] == 0) continue;
                if (begin[j] < so_far) S.bad = 1;
                so_far = max(so_far, begin[j] + n[j]);
                atomicMin(&S.first, begin[j]);
            }
            __syncthreads();   // S.end has been read
            if (tid == 0) S.end = max(S.end, all);
        }
        int total;
        int at = before + block_scan(sum, S.scan, total);
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
            const int i = tid * kRun + j;
            if (i < n_here) first[i] = at;
            at += n[j];
        }
        __syncthreads();
        return before + total;
    };
    {
        int tokens = 0;
        for (int s = 0; s < segs; ++s) tokens = load_entries(s, tokens, true);
        if (tid == 0) S.tokens = tokens;
    }
    cluster.sync();
    int n_tok = 0, base = 0, end = 0;
    bool bad = E > P.cap;
    for (int c = 0; c < C; ++c) {
        const Shared* o = cluster.map_shared_rank(&S, c);
        bad = bad || o->first < end;
        end = max(end, o->end);
        if (c < rank) base += o->tokens;
        n_tok += o->tokens;
        bad = bad || o->bad != 0;
    }
    const int count = min(n_tok, P.budget);
    const int pages = (count + kPage - 1) / kPage;
    bad = bad || DE < pages || DE > (LAZYATTN_MAX_START + 1) / kPage;
    int dst_bad = 0;
    for (int i = tid; i < min(DE, pages); i += kThreads)
        dst_bad |= (uint32_t)P.dst_entries[d0 + i] >= (uint32_t)pv.num_pages;
    bad = __syncthreads_or(dst_bad) != 0 || bad;
    if (bad && tid == 0) record_error(pv.status, LAZYATTN_ERANGE);
    const int cnt = bad ? 0 : count;

    // New entries: the upper word holds start, count and the writable bit (blocks of other
    // heads read the lower word, the page, meanwhile).
    if (h == 0 && rank == 0)
        for (int i = tid; i < DE; i += kThreads) {
            uint32_t* hi = reinterpret_cast<uint32_t*>(P.dst_entries + d0 + i) + 1;
            const uint32_t start = (uint32_t)min((int64_t)i * kPage, (int64_t)LAZYATTN_MAX_START);
            *hi = (*hi & 0x80000000u) | start | ((uint32_t)max(0, min(kPage, cnt - i * kPage)) << 26);
        }

    const int lo = min(P.sinks, n_tok), hi = max(lo, n_tok - P.recent);   // tokens [lo, hi) compete
    const bool all = cnt == n_tok;
    // The segment's keys: thread = (entry, 4 slots).
    auto load_keys = [&](int seg) {
        const int b0 = a0 + seg * P.seg, n_here = min(P.seg, a1 - b0);
#pragma unroll 4
        for (int x = tid; x < n_here * 4; x += kThreads) {
            const int i = x >> 2, s0 = (x & 3) * 4;
            const int n = min(entry_nvalid(P.entries[e0 + b0 + i]), kPage);
            const float4 m = *reinterpret_cast<const float4*>(P.mass + ((size_t)(e0 + b0 + i) * hkv + h) * kPage + s0);
            const int t = base + first[i] + s0;
            auto key = [&](float v, int j) {
                if (s0 + j >= n) return kNone;
                return all || t + j < lo || t + j >= hi ? kKeep : mass_key(v);
            };
            *reinterpret_cast<uint4*>(keys + x * 4) = make_uint4(key(m.x, 0), key(m.y, 1), key(m.z, 2), key(m.w, 3));
        }
        __syncthreads();
    };
    // Run f(slots) over the share with each segment's keys in place.
    auto each_segment = [&](auto f) {
        int before = 0;
        for (int s = 0; s < segs; ++s) {
            if (segs > 1) {
                __syncthreads();
                before = load_entries(s, before, false);
                load_keys(s);
            }
            f(min(P.seg, a1 - (a0 + s * P.seg)) * kPage);
        }
    };
    if (!bad && segs == 1) load_keys(0);

    uint32_t key = kNone;   // the smallest competing mass that stays (kNone: none does)
    int equal = 0;          // how many tokens equal to it stay
    int want = cnt - (n_tok - (hi - lo));   // of the competing tokens this many stay
    if (!bad && !all && want > 0) {
        key = 0;
#pragma unroll 1
        for (int dg = 0; dg < kDigits; ++dg) {
            const int shift = dg == 0 ? 21 : dg == 1 ? 10 : 0, bins = dg == 2 ? 1 << 10 : kBins;
            const uint32_t above = dg == 0 ? 0u : 0xffffffffu << (dg == 1 ? 21 : 10);   // the bits found so far
            each_segment([&](int slots) {
#pragma unroll 4
                for (int x = tid; x < slots; x += kThreads) {
                    const uint32_t k = keys[x];
                    if (k < kNone && (k & above) == key) atomicAdd(&S.hist[dg][(k >> shift) & (bins - 1)], 1);
                }
            });
            cluster.sync();
            // thread t has the bins 4 (511 - t) .. + 3, so that sums run from the largest masses down
            const int b0 = 4 * (kThreads - 1 - tid);
            int c4[4] = {0, 0, 0, 0};
            for (int c = 0; c < C; ++c) {
                const int4 v = *reinterpret_cast<const int4*>(cluster.map_shared_rank(&S, c)->hist[dg] + b0);
                c4[0] += v.x; c4[1] += v.y; c4[2] += v.z; c4[3] += v.w;
            }
            int total;
            int seen = block_scan(c4[0] + c4[1] + c4[2] + c4[3], S.scan, total);
#pragma unroll
            for (int j = 3; j >= 0; --j) {
                if (seen < want && want <= seen + c4[j]) {   // one thread, one bin
                    S.digit = b0 + j;
                    S.want = want - seen;
                }
                seen += c4[j];
            }
            __syncthreads();
            key |= (uint32_t)S.digit << shift;
            want = S.want;
            __syncthreads();
        }
        equal = want;
    }

    // A warp's contiguous part of a segment, 32 slots at a time: f(slot, kept for certain, equal to the threshold).
    auto each_slot = [&](int slots, auto f) {
        const int part = ((slots + 31) / 32 + kWarps - 1) / kWarps * 32;
        for (int x0 = warp * part; x0 < min(slots, (warp + 1) * part); x0 += 32) {
            const uint32_t k = x0 + lane < slots ? keys[x0 + lane] : kNone;
            f(x0 + lane, k == kKeep || (k < kNone && k > key), k < kNone && k == key);
        }
    };
    int sure = 0, same = 0;   // the warp's counts over the whole share
    if (!bad)
        each_segment([&](int slots) {
            each_slot(slots, [&](int, bool s, bool e) {
                sure += __popc(__ballot_sync(0xffffffffu, s));
                same += __popc(__ballot_sync(0xffffffffu, e));
            });
        });
    if (lane == 0) {
        S.warp_sure[warp] = sure;
        S.warp_equal[warp] = same;
    }
    __syncthreads();
    if (tid == 0) {
        int s = 0, e = 0;
        for (int w = 0; w < kWarps; ++w) {
            s += S.warp_sure[w];
            e += S.warp_equal[w];
        }
        S.sure = s;
        S.equal = e;
    }
    cluster.sync();
    int sure0 = 0, same0 = 0;   // tokens before this block's share (then: before the segment)
    for (int c = 0; c < rank; ++c) {
        const Shared* o = cluster.map_shared_rank(&S, c);
        sure0 += o->sure;
        same0 += o->equal;
    }
    // Places of the kept tokens, in table order. Of `same` tokens equal to the threshold the first
    // `equal` are kept, so the place of a token is (sure before) + min(equal, same before).
    if (!bad) {
        int at = 0;   // entries of the share before the segment
        each_segment([&](int slots) {
            if (segs > 1) {   // the warps' counts of this segment
                int s = 0, e = 0;
                each_slot(slots, [&](int, bool a, bool b) {
                    s += __popc(__ballot_sync(0xffffffffu, a));
                    e += __popc(__ballot_sync(0xffffffffu, b));
                });
                if (lane == 0) {
                    S.warp_sure[warp] = s;
                    S.warp_equal[warp] = e;
                }
                __syncthreads();
            }
            int s_at = sure0, e_at = same0;
            for (int w = 0; w < kWarps; ++w) {
                const int s = S.warp_sure[w], e = S.warp_equal[w];
                if (w < warp) {
                    s_at += s;
                    e_at += e;
                }
                sure0 += s;
                same0 += e;
            }
            each_slot(slots, [&](int x, bool s, bool e) {
                const unsigned below = (1u << lane) - 1u;
                const unsigned sb = __ballot_sync(0xffffffffu, s), eb = __ballot_sync(0xffffffffu, e);
                const int e_here = e_at + __popc(eb & below);
                if (s || (e && e_here < equal))
                    kept[s_at + __popc(sb & below) + min(equal, e_here)] = (a0 + at) * kPage + x;
                s_at += __popc(sb);
                e_at += __popc(eb);
            });
            at += P.seg;
        });
    }
    for (int64_t j = cnt + rank * kThreads + tid; j < P.budget; j += C * kThreads) kept[j] = -1;   // budgets up to 2^31 - 1
    const int used = (cnt + kPage - 1) / kPage * kPage;
    if (P.dst_mass)
        for (int64_t j = used + rank * kThreads + tid; j < (int64_t)DE * kPage; j += C * kThreads)
            P.dst_mass[((size_t)(d0 + j / kPage) * hkv + h) * kPage + j % kPage] = 0.f;
    cluster.sync();   // no block leaves while another reads its shared memory
}

// Block = (kept rows, KV head, request). A row's 16-byte vectors are consecutive threads of a
// warp; a place becomes the token's position once the block has read it. Slots of the
// last page past the tokens become zeros. One row a thread: more rows in flight per thread cost
// warps, which hide the three dependent loads better (32 requests cut to 2048 tokens, both kernels:
// 115 us; two rows 121, four 134, eight 244).
constexpr int kCopyThreads = 256;
template <int VECS>
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(PoolView pv, EvictParams P) {
    constexpr int kRows = kCopyThreads / VECS;
    const int h = blockIdx.y, r = blockIdx.z, hkv = pv.hkv;
    const int v = threadIdx.x % VECS, j = (int)blockIdx.x * kRows + (int)threadIdx.x / VECS;
    const int e0 = P.entry_offsets[r], d0 = P.dst_offsets[r];
    int32_t* kept = P.kept + ((size_t)r * hkv + h) * P.budget;
    uint4* kp = static_cast<uint4*>(pv.k_pool);
    uint4* vp = static_cast<uint4*>(pv.v_pool);
    grid_dep_wait();
    const int j16 = j / kPage * kPage;
    const int code = j < P.budget ? kept[j] : -1;
    const bool page = j16 < P.budget && kept[j16] >= 0;   // the row's page holds a kept token (place or position)
    __syncthreads();
    if (!page) return;
    const size_t slot = (size_t)j % kPage;
    const size_t dst = (((size_t)(uint32_t)P.dst_entries[d0 + j / kPage] * hkv + h) * kPage + slot) * VECS + v;
    uint4 a = make_uint4(0, 0, 0, 0), b = a;
    float m = 0.f;
    if (code >= 0) {
        const uint64_t e = P.entries[e0 + code / kPage];
        const size_t src = (((size_t)entry_page(e) * hkv + h) * kPage + code % kPage) * VECS + v;
        a = kp[src];
        b = vp[src];
        if (v == 0) {
            if (P.dst_mass) m = P.mass[((size_t)(e0 + code / kPage) * hkv + h) * kPage + code % kPage];
            kept[j] = entry_start(e) + code % kPage;
        }
    }
    kp[dst] = a;
    vp[dst] = b;
    if (v == 0 && P.dst_mass) P.dst_mass[((size_t)(d0 + j / kPage) * hkv + h) * kPage + slot] = m;
}

}  // namespace

// Blocks per (request, KV head). The phases are bound by their barriers and latencies, so
// blocks are few: one per 1024 entries (16 K tokens), or per 512 while all blocks fit the GPU
// at once (one request of 50,000 tokens: 24 us against 29; four: 48 against 39).
static int evict_cluster(const lazyattn_pool& p, const lazyattn_batch& b) {
    const int64_t items = (int64_t)b.num_requests * p.d.n_kv_heads;
    int c = 1;
    while (c < kMaxCluster && (b.max_entries > c * 1024 || (b.max_entries > c * 512 && items * 2 * c <= p.sm_count))) c *= 2;
    return c;
}

static int evict_smem(int seg) { return seg * (kPage * (int)sizeof(uint32_t) + (int)sizeof(int)); }

int evict_init() {
    return cudaFuncSetAttribute(evict_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, evict_smem(kSeg)) == cudaSuccess
               ? LAZYATTN_OK
               : LAZYATTN_ECUDA;
}

int launch_evict(const lazyattn_pool& p, const lazyattn_batch& b, const float* mass, int32_t budget, int32_t sinks,
                 int32_t recent, uint64_t* dst_entries, const int32_t* dst_offsets, int32_t* kept, float* dst_mass,
                 cudaStream_t stream) {
    const int C = evict_cluster(p, b);
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
    P.cap = b.max_entries;
    P.seg = std::min(kSeg, std::max(1, (b.max_entries + C - 1) / C));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(C, p.d.n_kv_heads, b.num_requests);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = evict_smem(P.seg);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = C;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, evict_kernel, p.view(), P) != cudaSuccess) return LAZYATTN_ECUDA;
    const bool wide = p.d.head_dim * (p.d.dtype == LAZYATTN_F32 ? 4 : 2) == 512;   // 16-byte vectors a row: 32, else 16
    const int rows = kCopyThreads / (wide ? 32 : 16);
    // A request keeps no more tokens than this, in whole pages: the blocks also write the empty slots behind the
    // last token, and a block of 512-byte rows is half a page.
    const int64_t most = (std::min<int64_t>(budget, (int64_t)b.max_entries * kPage) + kPage - 1) / kPage * kPage;
    if (most == 0) return LAZYATTN_OK;
    if (launch_dependent(wide ? evict_copy_kernel<32> : evict_copy_kernel<16>,
                         dim3((unsigned)((most + rows - 1) / rows), p.d.n_kv_heads, b.num_requests),
                         dim3(kCopyThreads), 0, stream, p.view(), P) != cudaSuccess)
        return LAZYATTN_ECUDA;
    return cudaGetLastError() == cudaSuccess ? LAZYATTN_OK : LAZYATTN_ECUDA;
}

}  // namespace lazyattn
