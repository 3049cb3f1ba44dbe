"""Windowed attention, attention mass and eviction: what is refused before any
CUDA call, and the reference's own rules - no GPU needed."""
import ctypes

import numpy as np
import pytest

import oracle
from tests.cache_common import attend


@pytest.fixture(scope="module")
def L():
    import __graft_entry__
    __graft_entry__.build()
    from position_agnostic_kv_lazyattn_gb300 import lazyattn
    return lazyattn


def test_null_handles_are_rejected(L):
    b = ctypes.byref(L.lazyattn_batch())
    assert L.lib.lazyattn_window_workspace_size(None, 0, b, 8, 0) == 0
    assert L.lib.lazyattn_prefill_window(None, b, None, None, 8, 0, None, 0, None) == -1
    assert L.lib.lazyattn_decode_window(None, b, None, None, None, None, 8, 0, None, 0, None) == -1
    assert L.lib.lazyattn_prefill_mass(None, b, None, None, None, 1.0, None, 0, None) == -1
    assert L.lib.lazyattn_decode_mass(None, b, None, None, None, None, None, None, 1.0, None, 0, None) == -1
    assert L.lib.lazyattn_evict(None, b, None, 8, 0, 0, None, None, None, None, None) == -1
    for call in (lambda: L.lib.lazyattn_decode_window(None, None, None, None, None, None, 8, 0, None, 0, None),
                 lambda: L.lib.lazyattn_decode_mass(None, None, None, None, None, None, None, None, 1.0, None, 0, None),
                 lambda: L.lib.lazyattn_evict(None, None, None, 8, 0, 0, None, None, None, None, None)):
        assert call() == -1


def test_strided_and_mistyped_tensors_are_rejected(L):
    import torch
    x = torch.zeros(4, 8)
    b = L.lazyattn_batch()
    for call in (lambda: L.lazyattn_prefill_window(0, b, x.t(), x, 8),
                 lambda: L.lazyattn_decode_window(0, b, x, x[:, ::2], x, x, 8, 0, x, 0),
                 lambda: L.lazyattn_prefill_mass(0, b, x, None, x.t(), 1.0, x, 0),
                 lambda: L.lazyattn_decode_mass(0, b, x, x, x, x, x.double(), x, 1.0, x, 0),
                 lambda: L.lazyattn_evict(0, b, x.double(), 8, 0, 0, x, x, x),
                 lambda: L.lazyattn_evict(0, b, x, 8, 0, 0, x.long(), x.int(), x.long())):
        with pytest.raises(L.LazyAttnError) as e:
            call()
        assert e.value.code == L.LAZYATTN_EINVAL


def test_the_reference_without_a_window_is_the_oracle():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((5, 4, 64)), rng.standard_normal((37, 2, 64)), rng.standard_normal((37, 2, 64))
    q_pos, k_pos = np.arange(32, 37), np.arange(37)
    for spec in (1e4, oracle.AlibiSpec()):
        ref = attend(spec, q, k, v, q_pos, k_pos)
        np.testing.assert_allclose(ref.out, oracle.attention(q, k, v, q_pos, k_pos, spec), atol=1e-12)
        np.testing.assert_allclose(ref.mass.sum(), 5 * 4, rtol=1e-12)


def test_the_reference_with_a_window_is_the_oracle_on_the_visible_tokens():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 4, 64)), rng.standard_normal((37, 2, 64)), rng.standard_normal((37, 2, 64))
    for window, sinks in [(1, 0), (5, 2), (100, 0), (4, 40)]:
        ref = attend(1e4, q, k, v, np.arange(34, 37), np.arange(37), window, sinks)
        for i, m in enumerate(range(34, 37)):
            see = np.array([n for n in range(m + 1) if m - n < window or n < sinks])
            np.testing.assert_allclose(ref.out[i], oracle.attention(q[i:i + 1], k[see], v[see], [m], see, 1e4)[0], atol=1e-12)


def test_short_and_misplaced_buffers_are_rejected(L, monkeypatch):
    """Tensors that a call would read or write past, read as another type, or find on another device: refused before the
    C library sees them (the handle is not one it could use)."""
    import torch
    bf, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    H, R, E, rows = 12345, 3, 7, 5
    shape = L._Shape(8 * 128, 2 * 128, 2, bf, -1)                       # "device" -1: where CPU tensors say they are
    monkeypatch.setitem(L._POOLS, H, shape)
    ent = torch.zeros(E, dtype=torch.int64)
    b = L.make_batch(R, 4, ent, torch.zeros(R + 1, dtype=i32), max_q_len=2, total_q=rows)
    assert b.n_entries == E and L.make_batch(R, 4, ent, None, n_entries=5).n_entries == 5

    def z(*dims, t=bf):
        return torch.zeros(*dims, dtype=t)

    q, q1, k1, m = z(rows, 8, 128), z(R, 8, 128), z(R, 2, 128), z(E, 2, 16, t=f32)
    kept, dst, off, ws = z(R, 2, 20, t=i32), z(6, t=torch.int64), z(R + 1, t=i32), z(256, t=torch.uint8)
    dm = z(6, 2, 16, t=f32)

    def window(q=q, out=q, ws=ws):
        L.lazyattn_prefill_window(H, b, q, out, 8, 0, ws, 256)

    def step(q=q1, k=k1, v=k1, out=q1, ws=ws):
        L.lazyattn_decode_window(H, b, q, k, v, out, 8, 0, ws, 256)

    def mass(q=q, old=m, new=m, ws=ws):
        L.lazyattn_prefill_mass(H, b, q, old, new, 1.0, ws, 256)

    def step_mass(q=q1, k=k1, v=k1, out=q1, old=m, new=m, ws=ws):
        L.lazyattn_decode_mass(H, b, q, k, v, out, old, new, 1.0, ws, 256)

    def evict(mass=m, dst=dst, off=off, kept=kept, dm=dm):
        L.lazyattn_evict(H, b, mass, 20, 0, 0, dst, off, kept, dm)

    calls = [
        lambda: window(q=q[:4]), lambda: window(out=q[:4]), lambda: window(q=q.float()), lambda: window(out=q.half()),
        lambda: window(ws=ws[:255]),
        lambda: step(q=q1[:2]), lambda: step(k=k1[:2]), lambda: step(v=k1.float()), lambda: step(out=q1[:, :7]),
        lambda: step(ws=ws[:255]),
        lambda: mass(q=q[:4]), lambda: mass(old=m[:6]), lambda: mass(new=m[:6]), lambda: mass(new=m.double()),
        lambda: mass(ws=ws[:255]),
        lambda: step_mass(q=q1[:2]), lambda: step_mass(k=k1.float()), lambda: step_mass(v=k1[:2]), lambda: step_mass(out=q1[:2]),
        lambda: step_mass(old=m[:6]), lambda: step_mass(new=m[:6]), lambda: step_mass(ws=ws[:255]),
        lambda: evict(mass=m[:6]), lambda: evict(off=off[:3]), lambda: evict(kept=kept[:, :, :19].contiguous()),
        lambda: evict(kept=kept[:2]), lambda: evict(dm=dm[:5]), lambda: evict(dst=dst.int()),
    ]
    for i, call in enumerate(calls):
        with pytest.raises(L.LazyAttnError) as e:
            call()
        assert e.value.code == L.LAZYATTN_EINVAL, i
    monkeypatch.setitem(L._POOLS, H, shape._replace(device=0))           # a pool on the GPU, tensors on the CPU
    for i, call in enumerate((window, step, mass, step_mass, evict)):
        with pytest.raises(L.LazyAttnError) as e:
            call()
        assert e.value.code == L.LAZYATTN_EINVAL, i
