// Windowed attention and attention mass of fp32 pools on CUDA cores, fp32 end to end
// (position-free or pre-rotated keys, rotary encodings; other layouts are bf16 only).
//
//   score(row, token) = log2(e) * scale * (R_m q) . (R_n k), log2 domain
//   out  = sum_n 2^(score - max) v_n / sum_n 2^(score - max)
//   mass = decay * mass_in + sum over rows and the group's heads of
//          2^(score - max_row) / sum_row
//
// Work on a page: lane = (slot, half of the head dim's pairs), so a warp scores the
// 16 keys of a page at once with one shuffle to join the halves; for the output,
// lane = dims and the 16 weights are broadcast by shuffles. Bound by latency at the sizes these
// pools serve (4 requests of ~900 tokens, 4/2 heads of 64: a step under a window of 300 takes 14 us in a graph of
// ten, 16 warps a block against 19 us with 4. As graphs of one pass, the copy that puts the table back with it:
// that step 18 us, a step with mass 33, 33 query rows a request under the window 33, their mass 94; heads of 128:
// 23, 51, 56 and 185). Each block reads its row's keys for itself.
#include "internal.h"

namespace lazyattn {

namespace {

constexpr int kWarps = 4;          // warps of a block
constexpr int kDecodeWarps = 16;   // of a decode step's, whose few blocks have a whole cache each
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }

struct Params {
    const uint64_t* entries;
    const int32_t* entry_offsets;
    const int32_t* q_offsets;     // prefill
    const int32_t* q_start;
    const int32_t* decode_qpos;   // decode: position of the appended token, -1 if none (else NULL)
    int32_t total_q;
    int32_t max_rows;             // prefill: rows per request that rows_kernel covers
    int32_t cap;                  // entries per request that take part (mass: the host's bound)
    int32_t window, sinks;
    int32_t causal;               // keys past the row's position are hidden
    int32_t rotate_k;             // 0: pre-rotated pages
    float2* stats;                // [row][Hq]: (largest score, 1 / sum), or NULL
    float* q_rot;                 // [row][Hq][D] rotated, scaled q, or NULL
};

__device__ __forceinline__ bool visible(const Params& P, int n, int m) {
    return !P.causal || (n <= m && (m - n < P.window || n < P.sinks));
}

// Entry's usable slots: 0 for an empty or an unusable one (reported).
__device__ __forceinline__ int slots_of(const PoolView& pv, uint64_t e) { return entry_ok(pv, e) ? entry_nvalid(e) : 0; }

// This lane's part of its key (slot lane % 16): D / 4 pairs from dim (lane / 16) * D / 4
// on, rotated to its position; x the first halves' dims, y their partners.
template <int D>
__device__ __forceinline__ void load_key(const PoolView& pv, const Params& P, const float* row, int pos, int d0,
                                         float (&x)[D / 4], float (&y)[D / 4]) {
#pragma unroll
    for (int j = 0; j < D / 4; j += 4) {
        const float4 a = load4(row + d0 + j), b = load4(row + d0 + j + D / 2);
        const float xs[4] = {a.x, a.y, a.z, a.w}, ys[4] = {b.x, b.y, b.z, b.w};
        if (P.rotate_k) {
            const float4* cs = reinterpret_cast<const float4*>(pv.rope + (size_t)pos * (D / 2) + d0 + j);
            const float4 c0 = cs[0], c1 = cs[1];
            const float co[4] = {c0.x, c0.z, c1.x, c1.z}, si[4] = {c0.y, c0.w, c1.y, c1.w};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                x[j + t] = xs[t] * co[t] - ys[t] * si[t];
                y[j + t] = xs[t] * si[t] + ys[t] * co[t];
            }
        } else {
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                x[j + t] = xs[t];
                y[j + t] = ys[t];
            }
        }
    }
}

template <int D>
__device__ __forceinline__ float dot_key(const float* q, int d0, const float (&x)[D / 4], const float (&y)[D / 4]) {
    float s = 0.f;
#pragma unroll
    for (int j = 0; j < D / 4; j += 4) {
        const float4 a = *reinterpret_cast<const float4*>(q + d0 + j);
        const float4 b = *reinterpret_cast<const float4*>(q + d0 + j + D / 2);
        s = fmaf(a.x, x[j], fmaf(a.y, x[j + 1], fmaf(a.z, x[j + 2], fmaf(a.w, x[j + 3], s))));
        s = fmaf(b.x, y[j], fmaf(b.y, y[j + 1], fmaf(b.z, y[j + 2], fmaf(b.w, y[j + 3], s))));
    }
    return s + __shfl_xor_sync(0xffffffffu, s, 16);
}

// Block = (query row, query head, request); its warps share the live entries.
// out NULL: statistics only.
template <int D, int kWarps>
__global__ void __launch_bounds__(kWarps * 32)
    rows_kernel(PoolView pv, Params P, const float* __restrict__ q, float* out) {
    constexpr int J = D / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.z, hq = blockIdx.y, i = blockIdx.x;
    const int kvh = hq / (pv.hq / pv.hkv);
    __shared__ __align__(16) float s_q[D];
    __shared__ float s_acc[kWarps][D], s_m[kWarps], s_l[kWarps];

    int row = r, m;
    if (P.decode_qpos) {
        m = P.decode_qpos[r];
    } else {
        const int q0 = P.q_offsets[r], q1 = P.q_offsets[r + 1];
        if (i >= q1 - q0) return;
        row = q0 + i;
        if (row >= P.total_q || q1 > P.total_q) {
            record_error(pv.status, LAZYATTN_ERANGE);
            return;
        }
        m = P.q_start[r] + i;
    }
    const size_t at = (size_t)row * pv.hq + hq;
    if (m < 0 || m >= pv.max_position) {
        if (m >= 0 || !P.decode_qpos) record_error(pv.status, LAZYATTN_ERANGE);
        if (out)
            for (int d = threadIdx.x; d < D; d += kWarps * 32) out[at * D + d] = 0.f;
        if (P.stats && threadIdx.x == 0) P.stats[at] = make_float2(0.f, 0.f);
        if (P.q_rot)   // never NaN, its weights are 0 by the statistics
            for (int d = threadIdx.x; d < D; d += kWarps * 32) P.q_rot[at * D + d] = 0.f;
        return;
    }
    for (int d = threadIdx.x; d < D / 2; d += kWarps * 32) {
        const float a = q[at * D + d], b = q[at * D + d + D / 2], sc = kLog2e * pv.qk_scale;
        const float2 cs = pv.rope[(size_t)m * (D / 2) + d];
        const float x = (a * cs.x - b * cs.y) * sc, y = (a * cs.y + b * cs.x) * sc;
        s_q[d] = x;
        s_q[d + D / 2] = y;
        if (P.q_rot) {
            P.q_rot[at * D + d] = x;
            P.q_rot[at * D + d + D / 2] = y;
        }
    }
    __syncthreads();

    const int slot = lane & 15, d0 = (lane >> 4) * (D / 4);
    const float* kpool = static_cast<const float*>(pv.k_pool);
    const float* vpool = static_cast<const float*>(pv.v_pool);
    float mx = -INFINITY, l = 0.f, acc[J];
#pragma unroll
    for (int j = 0; j < J; ++j) acc[j] = 0.f;
    const int e0 = P.entry_offsets[r], e1 = e0 + min(P.entry_offsets[r + 1] - e0, P.cap);
    int rank = 0;   // live entries before this chunk
    for (int c = e0; c < e1; c += 32) {
        const uint64_t mine = c + lane < e1 ? P.entries[c + lane] : 0ull;
        const int n_mine = c + lane < e1 ? slots_of(pv, mine) : 0;
        const int a = entry_start(mine), b = a + n_mine - 1;
        const bool live = n_mine > 0 && (!P.causal || (a <= m && (m - b < P.window || a < P.sinks)));
        unsigned todo = __ballot_sync(0xffffffffu, live);
        for (; todo; todo &= todo - 1, ++rank) {
            if (rank % kWarps != warp) continue;
            const int src = __ffs(todo) - 1;
            const uint64_t e = __shfl_sync(0xffffffffu, mine, src);
            const int n = __shfl_sync(0xffffffffu, n_mine, src);
            const int pos = entry_start(e) + slot;
            const bool see = slot < n && visible(P, pos, m);
            const size_t base = ((size_t)entry_page(e) * pv.hkv + kvh) * kPage * D;
            const int use = slot < n ? slot : 0;
            float x[D / 4], y[D / 4];
            load_key<D>(pv, P, kpool + base + (size_t)use * D, entry_start(e) + use, d0, x, y);
            float s = dot_key<D>(s_q, d0, x, y);
            s = see ? s : -INFINITY;
            float top = s;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            if (top == -INFINITY) continue;   // the page has tokens on both sides of the window, none inside
            const float mn = fmaxf(mx, top), corr = exp2f(mx - mn), p = exp2f(s - mn);
            float sum = p;
#pragma unroll
            for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            l = l * corr + sum;
            mx = mn;
            if (!out) continue;
#pragma unroll
            for (int j = 0; j < J; ++j) acc[j] *= corr;
#pragma unroll
            for (int t = 0; t < kPage; ++t) {
                const float pt = __shfl_sync(0xffffffffu, p, t);
                if (t < n) {
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        acc[j] = fmaf(pt, vpool[base + (size_t)t * D + lane + 32 * j], acc[j]);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) s_acc[warp][lane + 32 * j] = acc[j];
    if (lane == 0) {
        s_m[warp] = mx;
        s_l[warp] = l;
    }
    __syncthreads();
    float M = -INFINITY, L = 0.f;
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
    if (M != -INFINITY)
        for (int w = 0; w < kWarps; ++w) L += s_l[w] * exp2f(s_m[w] - M);
    const float inv = L > 0.f ? 1.f / L : 0.f;
    if (P.stats && threadIdx.x == 0) P.stats[at] = make_float2(M == -INFINITY ? 0.f : M, inv);
    if (out)
        for (int d = threadIdx.x; d < D; d += kWarps * 32) {
            float o = 0.f;
            if (M != -INFINITY)
                for (int w = 0; w < kWarps; ++w) o += s_acc[w][d] * exp2f(s_m[w] - M);
            out[at * D + d] = o * inv;
        }
}

// Warp = (entry, KV head, request): the mass of the entry's 16 slots over all rows.
template <int D>
__global__ void __launch_bounds__(kWarps * 32)
    mass_kernel(PoolView pv, Params P, const float* mass_in, float* mass_out, float decay) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = blockIdx.z, h = blockIdx.y;
    const int e0 = P.entry_offsets[r], E = P.entry_offsets[r + 1] - e0;
    if (E > P.cap && blockIdx.x == 0 && h == 0 && threadIdx.x == 0) record_error(pv.status, LAZYATTN_ERANGE);
    const int i = e0 + (int)blockIdx.x * kWarps + warp;
    if (i >= e0 + min(E, P.cap)) return;
    const int g = pv.hq / pv.hkv;
    const uint64_t e = P.entries[i];
    const int n = slots_of(pv, e);
    const int slot = lane & 15, d0 = (lane >> 4) * (D / 4);
    const int pos = entry_start(e) + slot;
    int row0, rows, m0;
    if (P.decode_qpos) {
        row0 = r;
        m0 = P.decode_qpos[r];
        rows = m0 >= 0 ? 1 : 0;
    } else {
        row0 = P.q_offsets[r];
        rows = min(P.q_offsets[r + 1] - row0, P.max_rows);
        m0 = P.q_start[r];
        if (P.q_offsets[r + 1] > P.total_q) rows = 0;   // reported by rows_kernel
    }
    float sum = 0.f;
    if (n > 0 && rows > 0) {
        const int use = slot < n ? slot : 0;
        const float* row = static_cast<const float*>(pv.k_pool) + (((size_t)entry_page(e) * pv.hkv + h) * kPage + use) * D;
        float x[D / 4], y[D / 4];
        load_key<D>(pv, P, row, entry_start(e) + use, d0, x, y);
        for (int t = 0; t < rows; ++t) {
            const int m = m0 + t;
            if (P.causal && m < entry_start(e)) continue;
            const bool see = slot < n && visible(P, pos, m);
            for (int j = 0; j < g; ++j) {
                const size_t at = (size_t)(row0 + t) * pv.hq + (size_t)h * g + j;
                const float2 st = P.stats[at];
                const float s = dot_key<D>(P.q_rot + at * D, d0, x, y);
                if (see) sum += exp2f(s - st.x) * st.y;
            }
        }
    }
    if (lane < kPage) {
        const size_t at = ((size_t)i * pv.hkv + h) * kPage + slot;
        float old = 0.f;
        if (mass_in && slot < n) old = rows == 0 && P.decode_qpos ? mass_in[at] : decay * mass_in[at];
        mass_out[at] = slot < n ? old + sum : 0.f;
    }
}

inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

Params make_params(const lazyattn_pool& p, const lazyattn_batch& b, const int32_t* decode_qpos, int32_t window,
                   int32_t sinks, bool causal) {
    Params P = {};
    P.entries = b.entries;
    P.entry_offsets = b.entry_offsets;
    P.q_offsets = b.q_offsets;
    P.q_start = b.q_start;
    P.decode_qpos = decode_qpos;
    P.total_q = decode_qpos ? b.num_requests : b.total_q;
    P.max_rows = b.max_q_len;
    P.cap = INT32_MAX;
    P.window = window;
    P.sinks = sinks;
    P.causal = causal;
    P.rotate_k = !(b.flags & LAZYATTN_KEYS_PREROTATED);
    return P;
}

int launch_rows(const lazyattn_pool& p, const lazyattn_batch& b, const Params& P, const void* q, void* out,
                cudaStream_t stream) {
    const int rows = P.decode_qpos ? 1 : b.max_q_len;
    if (rows < 1 || P.total_q < 1) return LAZYATTN_OK;
    const dim3 grid(rows, p.d.n_q_heads, b.num_requests);
    const int warps = P.decode_qpos ? kDecodeWarps : kWarps;
    auto k = P.decode_qpos ? (p.d.head_dim == 64 ? rows_kernel<64, kDecodeWarps> : rows_kernel<128, kDecodeWarps>)
                           : (p.d.head_dim == 64 ? rows_kernel<64, kWarps> : rows_kernel<128, kWarps>);
    k<<<grid, warps * 32, 0, stream>>>(p.view(), P, static_cast<const float*>(q), static_cast<float*>(out));
    return cudaGetLastError() == cudaSuccess ? LAZYATTN_OK : LAZYATTN_ECUDA;
}

int launch_mass(const lazyattn_pool& p, const lazyattn_batch& b, const Params& P, const float* mass_in, float* mass_out,
                float decay, cudaStream_t stream) {
    if (b.max_entries < 1) return LAZYATTN_OK;
    const dim3 grid((b.max_entries + kWarps - 1) / kWarps, p.d.n_kv_heads, b.num_requests);
    auto k = p.d.head_dim == 64 ? mass_kernel<64> : mass_kernel<128>;
    k<<<grid, kWarps * 32, 0, stream>>>(p.view(), P, mass_in, mass_out, decay);
    return cudaGetLastError() == cudaSuccess ? LAZYATTN_OK : LAZYATTN_ECUDA;
}

}  // namespace

int launch_window_simt(const lazyattn_pool& p, const lazyattn_batch& b, const void* q, void* out,
                       const int32_t* decode_qpos, int32_t window, int32_t sinks, cudaStream_t stream) {
    const Params P = make_params(p, b, decode_qpos, window, sinks, true);
    return launch_rows(p, b, P, q, out, stream);
}

size_t mass_simt_ws_bytes(const lazyattn_pool& p, int64_t rows) {
    const size_t n = (size_t)rows * (size_t)p.d.n_q_heads;
    return up256(n * sizeof(float2)) + up256(n * (size_t)p.d.head_dim * sizeof(float));
}

int launch_mass_simt(const lazyattn_pool& p, const lazyattn_batch& b, const void* q, void* out,
                     const int32_t* decode_qpos, const float* mass_in, float* mass_out, float decay, void* ws,
                     cudaStream_t stream) {
    Params P = make_params(p, b, decode_qpos, INT32_MAX, 0, decode_qpos == nullptr);
    P.cap = b.max_entries;
    P.stats = static_cast<float2*>(ws);
    P.q_rot = reinterpret_cast<float*>(static_cast<char*>(ws) +
                                       up256((size_t)P.total_q * (size_t)p.d.n_q_heads * sizeof(float2)));
    const int rc = launch_rows(p, b, P, q, out, stream);
    return rc != LAZYATTN_OK ? rc : launch_mass(p, b, P, mass_in, mass_out, decay, stream);
}

}  // namespace lazyattn
