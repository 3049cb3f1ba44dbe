"""Scenarios and the 64-bit reference of the operators that keep a cache small:
windowed attention, attention mass, eviction."""
import dataclasses

import numpy as np
import torch

import oracle
import workload
import workload.device

THETA = 1.0e4
MODES = ["rope", "alibi", "doc_local", "interleaved", "yarn", "prerotated"]
YARN = dict(kind="yarn", factor=4.0, original_max_position=256, low=1.0, high=32.0)


def spec_of(mode):
    if mode == "alibi":
        return oracle.AlibiSpec()
    if mode == "interleaved":
        return oracle.RopeSpec(THETA, pairing="interleaved")
    if mode == "yarn":
        return oracle.RopeSpec(THETA, YARN["kind"], YARN["factor"], YARN["original_max_position"], YARN["low"], YARN["high"])
    return THETA


class Scenario:
    """Requests of ragged documents and an own (writable) segment, in a pool.

    requests: per request (document lengths, own tokens, query rows); the query rows
    are the last of its tokens. spare: free pages behind the own segment. q_scale spreads the scores."""

    def __init__(self, L, requests, mode="rope", dtype="bf16", hq=8, hkv=2, d=128, spare=1, seed=0, q_scale=2.0, extra=0,
                 gap=0):
        self.rounded = mode in ("prerotated", "doc_local")   # keys stored rotated, in bf16
        self.L, self.mode, self.dtype, self.hq, self.hkv, self.d = L, mode, dtype, hq, hkv, d
        self.spec = spec_of(mode)
        rng = np.random.default_rng(seed)
        self.rng = rng
        n_pages = sum(sum(-(-n // 16) for n in docs) + -(-own // 16) + spare for docs, own, _ in requests)
        longest = max(sum(docs) + own + gap * len(docs) for docs, own, _ in requests)
        self.pool = L.DevicePool(2 * n_pages + extra + 2, hq, hkv, d, dtype, THETA, longest + 16 * spare + 16,
                                 key_storage="doc_local" if mode == "doc_local" else "position_free",
                                 rope_interleaved=mode == "interleaved", rope_scaling=YARN if mode == "yarn" else None,
                                 position_encoding="alibi" if mode == "alibi" else "rope")
        self.segments, self.k, self.v, self.pos = [], [], [], []
        for docs, own, _ in requests:
            segs, at, ks, vs, ps = [], 0, [], [], []
            for j, n in enumerate(list(docs) + [own]):
                k, v = self.normal(n, hkv, d), self.normal(n, hkv, d)
                pages = self.pool.store_doc(self.dev(k), self.dev(v)) if n else []
                last = j == len(docs)
                if last:
                    pages = list(pages) + self.pool.alloc_pages(spare)
                if pages:
                    segs.append(L.Segment(pages, at, n, writable=last))
                ks.append(k); vs.append(v); ps.append(at + np.arange(n))
                at += n + gap
            self.segments.append(segs)
            self.k.append(np.concatenate(ks)); self.v.append(np.concatenate(vs)); self.pos.append(np.concatenate(ps))
        self.rows = [r for _, _, r in requests]
        self.starts = [int(p[len(p) - r]) if r else 0 for p, r in zip(self.pos, self.rows)]
        self.batch = L.Batch(self.segments, self.rows, self.starts)
        if mode == "prerotated":
            dst = self.batch.entries_host.copy()
            fresh = np.array(self.pool.alloc_pages(len(dst)), np.uint64)
            dst = (dst & ~np.uint64(0xFFFFFFFF)) | fresh
            cuda = torch.from_numpy(dst.view(np.int64).copy()).cuda()
            L.lazyattn_materialize(self.pool.handle, self.batch.c, cuda)
            self.batch = self.batch.with_entries(dst, L.LAZYATTN_KEYS_PREROTATED)
        self.q = self.normal(sum(self.rows), hq, d) * q_scale if sum(self.rows) else np.zeros((0, hq, d), np.float32)

    def normal(self, *shape):
        x = self.rng.standard_normal(shape).astype(np.float32)
        return workload.round_bf16(x) if self.dtype == "bf16" else x

    def dev(self, x):
        return workload.device.to_device(np.ascontiguousarray(x), self.dtype)

    def empty(self, *shape):
        return torch.full(shape, float("nan"), dtype=self.pool.tdtype, device="cuda")

    def row_slice(self, r):
        a = sum(self.rows[:r])
        return slice(a, a + self.rows[r])

    def n_entries(self):
        return int(self.batch.offsets_host[-1])

    def mass_of(self, per_request):
        """Per-request [n][hkv] token weights laid out as [entries][hkv][16] (table order = token order)."""
        out = np.zeros((max(1, self.n_entries()), self.hkv, 16))
        ent = self.batch.entries.cpu().numpy().view(np.uint64)
        for r, w in enumerate(per_request):
            t = 0
            for i in range(self.batch.offsets_host[r], self.batch.offsets_host[r + 1]):
                n = oracle.unpack_entry(int(ent[i]))[2]
                out[i, :, :n] = w[t:t + n].T
                t += n
            assert t == len(w)
        return out


@dataclasses.dataclass
class Reference:
    out: np.ndarray      # [rows][Hq][D]
    spread: np.ndarray   # sum of p |v|, like out
    mass: np.ndarray     # [n][Hkv]
    reach: float         # largest sum |q_i k_i| of a score (ALiBi: or bias), in the log2 domain


def attend(spec, q, k, v, q_pos, k_pos, window=None, sinks=0, causal=True):
    """Attention of the rows and the weight each key gets, in 64 bits."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    q_pos, k_pos = np.asarray(q_pos, np.int64), np.asarray(k_pos, np.int64)
    rows, hq, d = q.shape
    hkv, g = k.shape[1], hq // k.shape[1]
    slopes = None
    if isinstance(spec, oracle.AlibiSpec):
        slopes, scale = oracle.alibi_slopes(hq), 1.0 / np.sqrt(d)
    else:
        q, k, scale = oracle.rope(q, q_pos[:, None], spec), oracle.rope(k, k_pos[:, None], spec), oracle.logit_scale(d, spec)
    n, m = k_pos[None], q_pos[:, None]
    see = n <= m if causal else np.ones((rows, len(k_pos)), bool)
    if window is not None:
        see = see & ((m - n < window) | (n < sinks))
    ref = Reference(np.zeros((rows, hq, d)), np.zeros((rows, hq, d)), np.zeros((len(k_pos), hkv)), 0.0)
    for h in range(hq):
        s = q[:, h] @ k[:, h // g].T * scale
        ref.reach = max(ref.reach, float((np.abs(q[:, h]) @ np.abs(k[:, h // g]).T).max(initial=0.0) * scale * 1.4427))
        if slopes is not None:
            s = s - slopes[h] * (m - n)
            ref.reach = max(ref.reach, float((slopes[h] * np.abs(m - n)).max(initial=0.0)) * 1.4427)
        s = np.where(see, s, -np.inf)
        top = s.max(1, keepdims=True, initial=-np.inf)
        p = np.where(see, np.exp(s - np.where(np.isfinite(top), top, 0.0)), 0.0)
        total = p.sum(1, keepdims=True)
        p = np.divide(p, total, out=np.zeros_like(p), where=total > 0)
        ref.out[:, h], ref.spread[:, h] = p @ v[:, h // g], p @ np.abs(v[:, h // g])
        ref.mass[:, h // g] += p.sum(0)
    return ref


def check_out(got, ref, dtype, rounded=False, row=slice(None)):
    """fp32 pools: max-abs 1e-4, as everywhere. bf16 pools, per element: the weights are rounded to bf16 for the product
    with V (half a step, 2^-8, of sum p |v|) and the output once more (2^-8 of it); a score's error is at most the fp16
    roundings of the rotated q and k (2^-11 each) of `reach`, and a weight and its row's sum each carry it, times ln 2.
    Keys stored rotated (`rounded`) were rounded to bf16 before (2^-8). In the norm these average out: 5e-3, as everywhere."""
    got, want, spread = np.asarray(got, np.float64), ref.out[row], ref.spread[row]
    assert got.shape == want.shape and np.all(np.isfinite(got))
    err = np.abs(got - want)
    if dtype == "f32":
        assert err.max(initial=0.0) <= 1e-4, err.max()
        return
    rel = 2.0 ** -8 + 2 * np.log(2) * ref.reach * (2.0 ** -10 + (2.0 ** -8 if rounded else 0.0))
    worst = np.max(err - rel * spread - 2.0 ** -8 * np.abs(want))
    assert worst <= 0, worst
    norm = np.linalg.norm(err) / max(np.linalg.norm(want), 1e-300)
    assert norm <= 5e-3, norm


def check_mass(got, want, reach, rounded=False):
    """A score's error (log2 units) is at most 72 steps of 2^-24 of the sum of its terms' sizes (`reach`): six roundings in
    the rotation of each operand, 12 in the split into two fp16 numbers (2^-22 each and for the dropped product) and 24
    accumulations that may truncate (2^-23 each). The weight and its row's sum each carry that error, times ln 2;
    2^-19 for the exponentials and the sums. Keys stored rotated (`rounded`: materialised or document-local pages) were
    rounded to bf16: half a step, 2^-8, per element."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape and np.all(np.isfinite(got))
    rel = 2 * np.log(2) * reach * (72 * 2.0 ** -24 + (2.0 ** -8 if rounded else 0.0)) + 2.0 ** -19
    worst = np.max(np.abs(got - want) - rel * want)
    assert worst <= 1e-30, (worst, rel)
