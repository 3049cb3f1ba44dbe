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
