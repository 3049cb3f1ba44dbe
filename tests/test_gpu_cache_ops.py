"""GPU tests of windowed attention, attention mass and eviction against the
64-bit definitions of tests/cache_common.py, on every key layout and position
encoding, with ragged tables and the sizes where such kernels go wrong."""
import numpy as np
import pytest
import torch

import oracle
from tests.cache_common import MODES, Scenario, attend, check_mass, check_out
from tests.gpu_common import compare

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def L():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    import __graft_entry__
    __graft_entry__.build()
    import position_agnostic_kv_lazyattn_gb300 as L
    return L


def workspace(L, s, op, window=None, sinks=0):
    n = (L.lazyattn_workspace_size(s.pool.handle, op, s.batch.c) if window is None else
         L.lazyattn_window_workspace_size(s.pool.handle, op, s.batch.c, window, sinks))
    assert n > 0
    return torch.zeros(n, dtype=torch.uint8, device="cuda"), n


def prefill_window(L, s, window, sinks):
    ws, n = workspace(L, s, L.LAZYATTN_OP_PREFILL, window, sinks)
    out = s.empty(max(1, s.batch.total_q), s.hq, s.d)
    L.lazyattn_prefill_window(s.pool.handle, s.batch.c, s.dev(s.q), out, window, sinks, ws, n)
    return out.float().cpu().numpy()


def check_prefill_window(L, s, window, sinks):
    got = prefill_window(L, s, window, sinks)
    for r, rows in enumerate(s.rows):
        if not rows:
            continue
        want = attend(s.spec, s.q[s.row_slice(r)], s.k[r], s.v[r], s.starts[r] + np.arange(rows), s.pos[r], window, sinks)
        check_out(got[s.row_slice(r)], want, s.dtype, s.rounded)
    assert s.pool.device_status() == 0


@pytest.mark.parametrize("mode", MODES)
def test_prefill_window_modes(L, mode):
    s = Scenario(L, [([70, 33], 40, 40), ([5, 100, 130], 17, 9), ([], 30, 30)], mode)
    check_prefill_window(L, s, 50, 3)


@pytest.mark.parametrize("hq,hkv", [(2, 2), (4, 2), (8, 2), (8, 1)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (17, 16), (100, 5), (128, 128), (1000, 0), (2**31 - 1, 0)])
def test_prefill_window_sizes(L, hq, hkv, window, sinks):
    """Windows of one token, of a page and around it, past the whole cache; odd lengths, a request without rows."""
    s = Scenario(L, [([260, 1, 16], 129, 129), ([40], 8, 0), ([], 1, 1), ([17, 300], 300, 130)], hq=hq, hkv=hkv, seed=1)
    check_prefill_window(L, s, window, sinks)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("window,sinks", [(1, 0), (20, 3), (10000, 0)])
def test_prefill_window_fp32(L, d, window, sinks):
    s = Scenario(L, [([70, 33], 40, 40), ([5, 100, 130], 17, 9), ([], 1, 1)], dtype="f32", hq=4, hkv=2, d=d, q_scale=1.0)
    check_prefill_window(L, s, window, sinks)


def test_prefill_window_long(L):
    """Many tiles, most of them skipped: rows in the middle and at the end of a long sequence."""
    s = Scenario(L, [([900] * 9, 200, 200), ([500, 500], 90, 90)], seed=2)
    for window, sinks in [(64, 4), (700, 0), (3000, 20)]:
        check_prefill_window(L, s, window, sinks)


def test_prefill_window_of_everything_is_prefill(L):
    s = Scenario(L, [([300, 33], 90, 90)], seed=3)
    out = s.empty(90, s.hq, s.d)
    L.lazyattn_prefill(s.pool.handle, s.batch.c, s.dev(s.q), out)
    got = prefill_window(L, s, 100000, 0)
    np.testing.assert_array_equal(got, out.float().cpu().numpy())


def test_prefill_window_rows_that_see_nothing(L):
    """Positions with gaps: rows whose window holds no token get zeros; entries out of order and empty ones."""
    s = Scenario(L, [([20, 50], 30, 30)], seed=4, gap=100)
    b = s.batch
    order = np.r_[np.arange(s.n_entries())[::-1]]
    ent = b.entries_host[order]
    b2 = b.with_entries(ent, 0)
    q = s.normal(64, s.hq, s.d) * 2
    start = 60                                     # positions 60..123: documents at 0..19 and 120..169
    off = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    qs = torch.tensor([start], dtype=torch.int32, device="cuda")
    c = L.lazyattn.make_batch(1, b.max_entries, b2.entries, b.entry_offsets, off, qs, 64, 64)
    out = s.empty(64, s.hq, s.d)
    L.lazyattn_prefill_window(s.pool.handle, c, s.dev(q), out, 30, 0)
    want = attend(s.spec, q, s.k[0], s.v[0], start + np.arange(64), s.pos[0], 30, 0)
    assert np.all(want.out[:60] == 0) and np.any(want.out[60:] != 0)
    got = out.float().cpu().numpy()
    assert np.all(got[:60] == 0)
    check_out(got, want, "bf16")


@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 2), (8, 1)])
@pytest.mark.parametrize("table", ["none", "empty entries", "before the window"])
def test_prefill_window_without_a_live_tile(L, hq, hkv, table):
    """No row of a request sees a key: no entries at all, entries without tokens, every token before the window (and past
    it: the sinks). Zeros in every row, whatever q holds, beside a request that does see keys."""
    s = Scenario(L, [([300], 10, 10)], hq=hq, hkv=hkv, seed=41)
    words = {"none": [], "empty entries": [L.pack_entries([0], [0], [0], [0])[0]] * 9,
             "before the window": list(s.batch.entries_host)}[table]
    n = 300                                                    # rows of the request that sees nothing, at 1000 and on
    ent = torch.from_numpy(np.array(words + list(s.batch.entries_host), np.uint64).view(np.int64).copy()).cuda()
    off = torch.tensor([0, len(words), len(words) + s.n_entries()], dtype=torch.int32, device="cuda")
    q_off = torch.tensor([0, n, n + 10], dtype=torch.int32, device="cuda")
    big = L.DevicePool(s.pool.num_pages, hq, hkv, 128, "bf16", 1.0e4, 1400)   # the same pages, a longer position table
    big.k_pool.copy_(s.pool.k_pool)
    big.v_pool.copy_(s.pool.v_pool)
    q_start = torch.tensor([1000, s.starts[0]], dtype=torch.int32, device="cuda")
    c = L.lazyattn.make_batch(2, max(len(words), s.n_entries()), ent, off, q_off, q_start, n, n + 10)
    q = np.concatenate([s.normal(n, hq, 128) * 2, s.q])
    want = attend(s.spec, s.q, s.k[0], s.v[0], s.starts[0] + np.arange(10), s.pos[0], 200, 0)
    for _ in range(20):
        out = s.empty(n + 10, hq, 128)
        L.lazyattn_prefill_window(big.handle, c, s.dev(q), out, 200, 0)
        got = out.float().cpu().numpy()
        assert np.all(got[:n] == 0)
        check_out(got[n:], want, "bf16")
    assert big.device_status() == 0


@pytest.mark.parametrize("mode", ["rope", "alibi"])
@pytest.mark.parametrize("start", [-3, 485])
def test_rows_out_of_range(L, mode, start):
    """Rows before position 0 or past the position table: zeros, no weight, reported; the others as ever."""
    s = Scenario(L, [([300, 100], 40, 8)], mode, seed=39, spare=2)
    top = s.pool.max_position                          # 440 + 32 + 16
    n = 8
    q = s.normal(n, s.hq, s.d) * 2
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    qs = torch.tensor([start], dtype=torch.int32, device="cuda")
    c = L.lazyattn.make_batch(1, s.batch.max_entries, s.batch.entries, s.batch.entry_offsets, off, qs, n, n)
    inside = [i for i in range(n) if 0 <= start + i < top]
    assert 0 < len(inside) < n
    out = s.empty(n, s.hq, s.d)
    L.lazyattn_prefill_window(s.pool.handle, c, s.dev(q), out, 90, 2)
    assert s.pool.device_status() == L.LAZYATTN_ERANGE
    got = out.float().cpu().numpy()
    ref = attend(s.spec, q[inside], s.k[0], s.v[0], start + np.array(inside), s.pos[0], 90, 2)
    check_out(got[inside], ref, "bf16")
    assert np.all(np.delete(got, inside, 0) == 0)
    size = L.lazyattn_workspace_size(s.pool.handle, L.LAZYATTN_OP_PREFILL_MASS, c)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    mass = torch.empty(s.n_entries(), s.hkv, 16, device="cuda")
    L.lazyattn_prefill_mass(s.pool.handle, c, s.dev(q), None, mass, 1.0, ws, size)
    assert s.pool.device_status() == L.LAZYATTN_ERANGE
    ref = attend(s.spec, q[inside], s.k[0], s.v[0], start + np.array(inside), s.pos[0])
    check_mass(mass.cpu().numpy(), s.mass_of([ref.mass]), ref.reach)


def decode_state(s):
    return [k.copy() for k in s.k], [v.copy() for v in s.v], [p.copy() for p in s.pos]


def step_inputs(s, R):
    return s.normal(R, s.hq, s.d) * 2, s.normal(R, s.hkv, s.d), s.normal(R, s.hkv, s.d)


@pytest.mark.parametrize("mode", MODES)
def test_decode_window_modes(L, mode):
    s = Scenario(L, [([70, 33], 40, 0), ([5, 100, 130], 15, 0), ([], 30, 0)], mode)
    check_decode_window(L, s, 50, 3, 3)


def check_decode_window(L, s, window, sinks, steps):
    R = len(s.rows)
    ws, n = workspace(L, s, L.LAZYATTN_OP_DECODE, window, sinks)
    k, v, pos = decode_state(s)
    for _ in range(steps):
        q, kn, vn = step_inputs(s, R)
        out = s.empty(R, s.hq, s.d)
        L.lazyattn_decode_window(s.pool.handle, s.batch.c, s.dev(q), s.dev(kn), s.dev(vn), out, window, sinks, ws, n)
        got = out.float().cpu().numpy()
        for r in range(R):
            m = int(pos[r][-1]) + 1 if len(pos[r]) else 0
            k[r], v[r], pos[r] = np.r_[k[r], kn[r][None]], np.r_[v[r], vn[r][None]], np.r_[pos[r], m]
            want = attend(s.spec, q[r][None], k[r], v[r], [m], pos[r], window, sinks)
            check_out(got[r], want, s.dtype, s.rounded, 0)
            if window == 1 and sinks == 0:   # its own value, bit for bit
                np.testing.assert_array_equal(got[r], np.repeat(vn[r], s.hq // s.hkv, 0))
    assert s.pool.device_status() == 0


@pytest.mark.parametrize("hq,hkv", [(2, 2), (6, 2), (8, 2), (8, 1), (10, 2)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 0), (17, 16), (100, 5), (1000, 0), (2**31 - 1, 7)])
def test_decode_window_sizes(L, hq, hkv, window, sinks):
    s = Scenario(L, [([260, 1, 16], 129, 0), ([], 0, 0), ([], 1, 0), ([17, 300], 300, 0), ([], 16, 0)], hq=hq, hkv=hkv, seed=5)
    check_decode_window(L, s, window, sinks, 2)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_window_fp32(L, d):
    s = Scenario(L, [([70, 33], 40, 0), ([5, 400, 130], 17, 0), ([], 0, 0)], dtype="f32", hq=4, hkv=2, d=d)
    check_decode_window(L, s, 90, 3, 2)


@pytest.mark.parametrize("window,sinks", [(64, 4), (2500, 0), (5000, 300)])
def test_decode_window_long(L, window, sinks):
    s = Scenario(L, [([900] * 9, 200, 0), ([500, 500], 90, 0)], seed=6, hq=32, hkv=8)
    check_decode_window(L, s, window, sinks, 1)


def test_windows_do_not_read_what_they_hide(L):
    """Pages none of whose tokens is visible may hold anything."""
    s = Scenario(L, [([320, 320], 64, 20)], seed=7)
    hidden = [p for p in s.segments[0][0].pages[1:]] + [p for p in s.segments[0][1].pages[:10]]
    at = torch.tensor(hidden, device="cuda")
    s.pool.k_pool[at] = float("nan")
    s.pool.v_pool[at] = float("inf")
    check_prefill_window(L, s, 100, 16)
    check_decode_window(L, s, 100, 16, 1)


@pytest.mark.parametrize("delta", [-1, 65])
@pytest.mark.parametrize("window,sinks", [(9, 0), (9, 3), (25, 0), (1000, 0)])
def test_decode_window_with_a_bad_document_offset(L, delta, window, sinks):
    """The entry that the step's token would go into has an offset outside its document: reported, the entry takes no part,
    and q stands where the token would have: windows that end right behind a page's last token leave that page out."""
    s = Scenario(L, [([64], 8, 0)], "doc_local", seed=44)
    s.batch.entry_delta[4] = delta
    ws, n = workspace(L, s, L.LAZYATTN_OP_DECODE, window, sinks)
    q, kn, vn = step_inputs(s, 1)
    out = s.empty(1, s.hq, s.d)
    L.lazyattn_decode_window(s.pool.handle, s.batch.c, s.dev(q), s.dev(kn), s.dev(vn), out, window, sinks, ws, n)
    assert s.pool.device_status() == L.LAZYATTN_ERANGE
    want = attend(s.spec, q[0][None], s.k[0][:64], s.v[0][:64], [72], np.arange(64), window, sinks)
    check_out(out.float().cpu().numpy()[0], want, "bf16", True, 0)


def test_decode_window_without_a_slot(L):
    """A request with no writable free slot: zeros, reported; the others are served."""
    s = Scenario(L, [([40], 16, 0), ([20], 5, 0)], spare=0, seed=8)
    ws, n = workspace(L, s, L.LAZYATTN_OP_DECODE, 30, 2)
    q, kn, vn = step_inputs(s, 2)
    out = s.empty(2, s.hq, s.d)
    L.lazyattn_decode_window(s.pool.handle, s.batch.c, s.dev(q), s.dev(kn), s.dev(vn), out, 30, 2, ws, n)
    got = out.float().cpu().numpy()
    assert np.all(got[0] == 0)
    want = attend(s.spec, q[1][None], np.r_[s.k[1], kn[1][None]], np.r_[s.v[1], vn[1][None]], [25], np.arange(26), 30, 2)
    check_out(got[1], want, "bf16", row=0)
    assert s.pool.device_status() == L.LAZYATTN_ENODECODE


# ------------------------------------------------------------------------------------------------ mass

def check_prefill_mass(L, s, decay, old):
    rng = np.random.default_rng(11)
    ws, n = workspace(L, s, L.LAZYATTN_OP_PREFILL_MASS)
    before = [rng.random((len(p), s.hkv)).astype(np.float32) for p in s.pos] if old else None
    mass_in = torch.from_numpy(s.mass_of(before).astype(np.float32)).cuda() if old else None
    out = torch.full((s.n_entries() + 1, s.hkv, 16), float("nan"), device="cuda")
    q = s.dev(s.q) if len(s.q) else None
    L.lazyattn_prefill_mass(s.pool.handle, s.batch.c, q, mass_in, out, decay, ws, n)
    assert bool(torch.isnan(out[-1]).all())                                    # behind the table: left alone
    want, reach = [], 0.0
    for r, rows in enumerate(s.rows):
        ref = attend(s.spec, s.q[s.row_slice(r)], s.k[r], s.v[r], s.starts[r] + np.arange(rows), s.pos[r])
        want.append(ref.mass + (np.float32(decay) * before[r].astype(np.float64) if old else 0.0))
        reach = max(reach, ref.reach)
    check_mass(out[:-1].cpu().numpy(), s.mass_of(want), reach, s.rounded)
    again = torch.full_like(out, float("nan"))
    L.lazyattn_prefill_mass(s.pool.handle, s.batch.c, q, mass_in, again, decay, ws, n)
    assert torch.equal(out[:-1], again[:-1])                                   # equal calls, equal bits
    if old:                                                                    # in place
        L.lazyattn_prefill_mass(s.pool.handle, s.batch.c, q, mass_in, mass_in, decay, ws, n)
        assert torch.equal(out[:-1], mass_in)
    assert s.pool.device_status() == 0


@pytest.mark.parametrize("mode", MODES)
def test_prefill_mass_modes(L, mode):
    s = Scenario(L, [([70, 33], 40, 40), ([5, 100, 130], 17, 9), ([], 30, 30)], mode, seed=12)
    check_prefill_mass(L, s, 0.5, True)


@pytest.mark.parametrize("hq,hkv", [(2, 2), (6, 2), (8, 2), (8, 1), (10, 2)])
@pytest.mark.parametrize("rows", [1, 3, 64, 130, 300])
def test_prefill_mass_sizes(L, hq, hkv, rows):
    s = Scenario(L, [([260, 1, 16], rows, rows), ([40], 8, 0), ([], 1, 1), ([17, 300], 300, max(1, rows // 2))], hq=hq, hkv=hkv,
                 seed=13)
    check_prefill_mass(L, s, 1.0, rows != 3)


@pytest.mark.parametrize("d", [64, 128])
def test_prefill_mass_fp32(L, d):
    s = Scenario(L, [([70, 33], 40, 40), ([5, 100, 130], 17, 9), ([], 1, 1)], dtype="f32", hq=4, hkv=2, d=d, seed=14)
    check_prefill_mass(L, s, 0.9, True)


def test_prefill_mass_long(L):
    s = Scenario(L, [([900] * 9, 100, 100), ([500, 500], 90, 33)], seed=15, hq=8, hkv=2)
    check_prefill_mass(L, s, 1.0, False)


@pytest.mark.parametrize("down", [6, 10, 14])
def test_mass_of_small_keys_under_large_queries(L, down):
    """Keys scaled down and queries up by 2^down: the two fp16 numbers of a key component below 1/8 are exact to 2^-25, so a
    score is off by that times the sum of its query's components (as they enter the product), beside what
    check_mass counts."""
    s = Scenario(L, [([260, 40], 33, 33)], seed=53, q_scale=2.0 ** (down + 1))
    s.pool.k_pool *= 2.0 ** -down
    s.k[0] *= 2.0 ** -down
    ref = attend(s.spec, s.q, s.k[0], s.v[0], s.starts[0] + np.arange(33), s.pos[0])
    # a rotation at most sqrt(2) up in the sum of a pair's components
    reach = float(np.abs(s.q).sum(-1).max()) * np.sqrt(2.0) * 1.4427 / np.sqrt(128)
    ws, n = workspace(L, s, L.LAZYATTN_OP_PREFILL_MASS)
    out = torch.full((s.n_entries(), s.hkv, 16), float("nan"), device="cuda")
    L.lazyattn_prefill_mass(s.pool.handle, s.batch.c, s.dev(s.q), None, out, 1.0, ws, n)
    assert s.pool.device_status() == 0
    rel = 2 * np.log(2) * (ref.reach * 72 * 2.0 ** -24 + reach * 2.0 ** -25) + 2.0 ** -19
    got, want = out.cpu().numpy().astype(np.float64), s.mass_of([ref.mass])
    assert np.all(np.abs(got - want) <= rel * want + 1e-30), (np.max(np.abs(got - want) / np.maximum(want, 1e-30)), rel)


def test_prefill_mass_in_chunks_of_rows(L):
    """Rows observed a chunk at a time, each onto the last one's mass: what one call over all of them gives, in a
    workspace of one chunk."""
    s = Scenario(L, [([500, 77], 256, 256)], seed=54, hq=8, hkv=2)
    whole = workspace(L, s, L.LAZYATTN_OP_PREFILL_MASS)
    q = s.dev(s.q)
    before = np.random.default_rng(55).random((len(s.pos[0]), s.hkv)).astype(np.float32)
    old = torch.from_numpy(s.mass_of([before]).astype(np.float32)).cuda()
    mass = torch.full_like(old, float("nan"))
    off = torch.tensor([0, 64], dtype=torch.int32, device="cuda")
    for i in range(4):
        start = torch.tensor([s.starts[0] + 64 * i], dtype=torch.int32, device="cuda")
        c = L.lazyattn.make_batch(1, s.batch.max_entries, s.batch.entries, s.batch.entry_offsets, off, start, 64, 64)
        n = L.lazyattn_workspace_size(s.pool.handle, L.LAZYATTN_OP_PREFILL_MASS, c)
        assert 0 < n < whole[1]
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        L.lazyattn_prefill_mass(s.pool.handle, c, q[64 * i:64 * i + 64], old if i == 0 else mass, mass, 0.5 if i == 0 else 1.0, ws, n)
    ref = attend(s.spec, s.q, s.k[0], s.v[0], s.starts[0] + np.arange(256), s.pos[0])
    check_mass(mass.cpu().numpy(), s.mass_of([ref.mass + 0.5 * before.astype(np.float64)]), ref.reach)
    assert s.pool.device_status() == 0


def test_prefill_mass_without_rows(L):
    """No row at all: the weights fade, nothing is added."""
    s = Scenario(L, [([70, 33], 40, 0), ([], 3, 0)], seed=16)
    s.batch.q_offsets = torch.zeros(3, dtype=torch.int32, device="cuda")
    s.batch.q_start = torch.zeros(2, dtype=torch.int32, device="cuda")
    s.batch.c.q_offsets, s.batch.c.q_start = s.batch.q_offsets.data_ptr(), s.batch.q_start.data_ptr()
    check_prefill_mass(L, s, 0.25, True)


def check_decode_mass(L, s, decay, steps, spare_mass=True):
    R = len(s.rows)
    ws, n = workspace(L, s, L.LAZYATTN_OP_DECODE_MASS)
    k, v, pos = decode_state(s)
    mass = torch.zeros(s.n_entries() + 1, s.hkv, 16, device="cuda") if spare_mass else None
    total = [np.zeros((len(p), s.hkv)) for p in pos]
    reach = 0.0
    for _ in range(steps):
        q, kn, vn = step_inputs(s, R)
        out = s.empty(R, s.hq, s.d)
        new = torch.full((s.n_entries() + 1, s.hkv, 16), float("nan"), device="cuda") if not spare_mass else mass
        L.lazyattn_decode_mass(s.pool.handle, s.batch.c, s.dev(q), s.dev(kn), s.dev(vn), out, mass, new, decay, ws, n)
        got = out.float().cpu().numpy()
        for r in range(R):
            m = int(pos[r][-1]) + 1 if len(pos[r]) else 0
            k[r], v[r], pos[r] = np.r_[k[r], kn[r][None]], np.r_[v[r], vn[r][None]], np.r_[pos[r], m]
            want = attend(s.spec, q[r][None], k[r], v[r], [m], pos[r], causal=False)
            reach = max(reach, want.reach)
            check_out(got[r], want, s.dtype, s.rounded, 0)
            total[r] = (decay * np.r_[total[r], np.zeros((1, s.hkv))] if spare_mass else 0.0) + want.mass
        check_mass(new[:-1].cpu().numpy(), s.mass_of(total), reach, s.rounded)
    assert s.pool.device_status() == 0


@pytest.mark.parametrize("mode", MODES)
def test_decode_mass_modes(L, mode):
    s = Scenario(L, [([70, 33], 40, 0), ([5, 100, 130], 15, 0), ([], 30, 0)], mode, seed=17)
    check_decode_mass(L, s, 0.5, 3)


@pytest.mark.parametrize("hq,hkv", [(2, 2), (6, 2), (8, 2), (8, 1), (10, 2)])
@pytest.mark.parametrize("decay,old", [(1.0, True), (0.0, False)])
def test_decode_mass_sizes(L, hq, hkv, decay, old):
    s = Scenario(L, [([260, 1, 16], 129, 0), ([], 0, 0), ([], 1, 0), ([17, 300], 300, 0), ([], 16, 0)], hq=hq, hkv=hkv, seed=18)
    check_decode_mass(L, s, decay, 2, old)


@pytest.mark.parametrize("d", [64, 128])
def test_decode_mass_fp32(L, d):
    s = Scenario(L, [([70, 33], 40, 0), ([5, 400, 130], 17, 0), ([], 0, 0)], dtype="f32", hq=4, hkv=2, d=d, seed=19)
    check_decode_mass(L, s, 1.0, 2)


def test_decode_mass_long(L):
    s = Scenario(L, [([900] * 9, 200, 0), ([500, 500], 90, 0)], seed=20, hq=32, hkv=8)
    check_decode_mass(L, s, 1.0, 2)


def test_decode_mass_output_is_decode(L):
    """The same output as a plain decode step, to the bounds of both."""
    outs = []
    for which in range(2):
        s = Scenario(L, [([260, 1, 16], 129, 0), ([17, 300], 300, 0)], seed=21)
        q, kn, vn = step_inputs(s, 2)
        out = s.empty(2, s.hq, s.d)
        if which:
            ws, n = workspace(L, s, L.LAZYATTN_OP_DECODE_MASS)
            mass = torch.empty(s.n_entries(), s.hkv, 16, device="cuda")
            L.lazyattn_decode_mass(s.pool.handle, s.batch.c, s.dev(q), s.dev(kn), s.dev(vn), out, None, mass, 1.0, ws, n)
        else:
            ws, n = workspace(L, s, L.LAZYATTN_OP_DECODE)
            L.lazyattn_decode(s.pool.handle, s.batch.c, s.dev(q), s.dev(kn), s.dev(vn), out, ws, n)
        outs.append(out.float().cpu().numpy())
    compare(outs[1], outs[0], "bf16")


def test_decode_mass_without_a_slot(L):
    """A request with no writable free slot keeps its mass, unfaded."""
    s = Scenario(L, [([40], 16, 0), ([20], 5, 0)], spare=0, seed=22)
    ws, n = workspace(L, s, L.LAZYATTN_OP_DECODE_MASS)
    q, kn, vn = step_inputs(s, 2)
    out = s.empty(2, s.hq, s.d)
    before = s.mass_of([np.full((56, s.hkv), 0.75), np.full((25, s.hkv), 0.5)]).astype(np.float32)
    mass = torch.from_numpy(before).cuda()
    L.lazyattn_decode_mass(s.pool.handle, s.batch.c, s.dev(q), s.dev(kn), s.dev(vn), out, mass, mass, 0.5, ws, n)
    got = mass.cpu().numpy()
    np.testing.assert_array_equal(got[:4], before[:4])
    assert np.all(out[0].float().cpu().numpy() == 0)
    ref = attend(s.spec, q[1][None], np.r_[s.k[1], kn[1][None]], np.r_[s.v[1], vn[1][None]], [25], np.arange(26))
    check_mass(got, s.mass_of([np.full((56, s.hkv), 0.75), ref.mass + 0.25 * (np.arange(26) < 25)[:, None]]), ref.reach)
    assert s.pool.device_status() == L.LAZYATTN_ENODECODE


# ------------------------------------------------------------------------------------------------ eviction

def kept_tokens(w, budget, sinks, recent):
    """Token numbers one head keeps, from its tokens' weights: sorted by (weight, NaN least; earlier first)."""
    n = len(w)
    if n <= budget:
        return np.arange(n)
    fixed = np.r_[np.arange(min(sinks, n)), np.arange(max(min(sinks, n), n - recent), n)]
    free = np.setdiff1d(np.arange(n), fixed)
    key = np.where(np.isnan(w), -np.inf, w)
    nan = np.isnan(w)
    best = sorted(free, key=lambda t: (nan[t], -key[t], t))[: budget - len(fixed)]
    return np.sort(np.r_[fixed, best]).astype(int)


def check_evict(L, s, weights, budget, sinks, recent, spare=1, dst_mass=True):
    R = len(s.rows)
    per = -(-budget // 16) + spare
    pages = np.array(s.pool.alloc_pages(R * per))
    wr = np.zeros(R * per, int)
    wr[1::2] = 1
    dst = torch.from_numpy(L.pack_entries(pages, np.full(R * per, 77), np.full(R * per, 9), wr).view(np.int64).copy()).cuda()
    off = torch.arange(R + 1, dtype=torch.int32, device="cuda") * per
    mass = torch.from_numpy(s.mass_of(weights).astype(np.float32)).cuda()
    kept = torch.full((R + 1, s.hkv, budget), -7, dtype=torch.int32, device="cuda")
    out_mass = torch.full((R * per + 1, s.hkv, 16), float("nan"), device="cuda") if dst_mass else None
    at = torch.from_numpy(pages).cuda()
    s.pool.k_pool[at] = 3.0
    s.pool.v_pool[at] = 3.0
    k0, v0 = s.pool.k_pool.clone(), s.pool.v_pool.clone()
    L.lazyattn_evict(s.pool.handle, s.batch.c, mass, budget, sinks, recent, dst, off, kept, out_mass)
    assert s.pool.device_status() == 0
    kept, dst_h = kept.cpu().numpy(), dst.cpu().numpy().view(np.uint64)
    assert np.all(kept[R] == -7)
    want_k, want_v = k0.clone(), v0.clone()
    want_mass = np.zeros((R * per, s.hkv, 16), np.float32)
    ent = s.batch.entries.cpu().numpy().view(np.uint64)
    for r in range(R):
        toks = oracle.resolve_entries(ent[s.batch.offsets_host[r]:s.batch.offsets_host[r + 1]])
        count = min(len(toks), budget)
        for i in range(per):
            assert oracle.unpack_entry(int(dst_h[r * per + i])) == (pages[r * per + i], 16 * i, max(0, min(16, count - 16 * i)),
                                                                      wr[r * per + i])
        for h in range(s.hkv):
            ids = kept_tokens(np.asarray(weights[r])[:, h].astype(np.float32), budget, sinks, recent)
            assert len(ids) == count
            want = np.full(budget, -1)
            want[:count] = [toks[t][2] for t in ids]
            np.testing.assert_array_equal(kept[r, h], want)
            for j in range(-(-count // 16) * 16):
                p, slot = int(pages[r * per + j // 16]), j % 16
                if j < count:
                    src = toks[ids[j]]
                    want_k[p, h, slot], want_v[p, h, slot] = k0[src[0], h, src[1]], v0[src[0], h, src[1]]
                    want_mass[r * per + j // 16, h, slot] = weights[r][ids[j], h]
                else:
                    want_k[p, h, slot] = want_v[p, h, slot] = 0
    assert torch.equal(s.pool.k_pool, want_k) and torch.equal(s.pool.v_pool, want_v)   # and nothing else was written
    if dst_mass:
        np.testing.assert_array_equal(out_mass[:-1].cpu().numpy(), want_mass)
        assert bool(torch.isnan(out_mass[-1]).all())


def weights_of(s, kind, rng):
    ws = []
    for p in s.pos:
        w = rng.standard_normal((len(p), s.hkv)).astype(np.float32)
        if kind == "ties":
            w = np.round(np.exp(w)).astype(np.float32)
        if kind == "equal":
            w[:] = 0.25
        if kind == "odd":   # NaN, infinities, both zeros, denormals
            w = np.array([np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42, -1e-42, 1.0, -1.0], np.float32)[rng.integers(0, 9, w.shape)]
        ws.append(w)
    return ws


@pytest.mark.parametrize("kind", ["normal", "ties", "equal", "odd"])
@pytest.mark.parametrize("budget,sinks,recent", [(1, 0, 0), (1, 0, 1), (16, 0, 0), (50, 4, 10), (33, 33, 0), (100, 0, 100), (500, 3, 9)])
def test_evict(L, kind, budget, sinks, recent):
    s = Scenario(L, [([70, 33], 40, 0), ([5, 100, 130], 17, 0), ([], 1, 0), ([], 0, 0)], seed=23, extra=4 * 34)
    check_evict(L, s, weights_of(s, kind, np.random.default_rng(24)), budget, sinks, recent)


@pytest.mark.parametrize("dtype,hq,hkv,d,mode", [("f32", 4, 2, 64, "rope"), ("f32", 4, 2, 128, "rope"), ("bf16", 8, 8, 128, "alibi"),
                                                 ("bf16", 6, 3, 128, "interleaved"), ("bf16", 8, 1, 128, "yarn")])
def test_evict_pools(L, dtype, hq, hkv, d, mode):
    s = Scenario(L, [([70, 33], 40, 0), ([5, 100, 130], 17, 0)], mode, dtype, hq, hkv, d, seed=25, extra=40)
    check_evict(L, s, weights_of(s, "normal", np.random.default_rng(26)), 61, 4, 10, dst_mass=False)


@pytest.mark.parametrize("dtype,d", [("f32", 64), ("f32", 128), ("bf16", 128)])
@pytest.mark.parametrize("budget", [5, 16, 50, 56, 57, 63])
def test_evict_budgets_that_end_inside_a_page(L, dtype, d, budget):
    """The rest of the last page: zeros, and no mass, for every size of a row."""
    s = Scenario(L, [([70, 33], 40, 0), ([5, 100, 130], 17, 0), ([], 3, 0)], dtype=dtype, hq=4, hkv=2, d=d, seed=42, extra=40)
    check_evict(L, s, weights_of(s, "normal", np.random.default_rng(43)), budget, 2, 3)


def test_a_cut_cache_of_wide_rows_goes_on_observing(L):
    """fp32, 512-byte rows, a budget that ends inside a page: the step after appends into that page, and its tokens' mass
    starts from 0."""
    s = Scenario(L, [([70, 33], 40, 0), ([5, 100, 130], 17, 0)], dtype="f32", hq=4, hkv=2, d=128, seed=46, extra=20)
    w = [np.abs(x) for x in weights_of(s, "normal", np.random.default_rng(47))]
    budget = 50
    at = torch.tensor(s.pool.alloc_pages(10), device="cuda")      # what the new pages held before
    s.pool.k_pool[at] = s.pool.v_pool[at] = float("nan")
    s.pool.free_pages(at.tolist())
    junk = torch.full((10, s.hkv, 16), float("nan"), device="cuda")   # and the block that new_mass may be given
    del junk
    mass = torch.from_numpy(s.mass_of(w).astype(np.float32)).cuda()
    batch, kept, mass = s.batch.evict(s.pool, mass, budget, sinks=2, recent=3)
    n = L.lazyattn_workspace_size(s.pool.handle, L.LAZYATTN_OP_DECODE_MASS, batch.c)
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    q, kn, vn = step_inputs(s, 2)
    out = s.empty(2, s.hq, s.d)
    L.lazyattn_decode_mass(s.pool.handle, batch.c, s.dev(q), s.dev(kn), s.dev(vn), out, mass, mass, 1.0, ws, n)
    got = mass.cpu().numpy().reshape(2, 5, s.hkv, 16).transpose(0, 2, 1, 3).reshape(2, s.hkv, 80)
    for r in range(2):
        for h in range(s.hkv):
            ids = kept_tokens(w[r][:, h], budget, 2, 3)
            k, v = np.r_[s.k[r][ids, h], kn[r, h][None]], np.r_[s.v[r][ids, h], vn[r, h][None]]
            ref = attend(s.spec, q[r, 2 * h:2 * h + 2][None], k[:, None], v[:, None], [budget], np.arange(budget + 1))
            check_out(out[r, 2 * h:2 * h + 2].cpu().numpy(), ref, "f32", row=0)
            check_mass(got[r, h, :budget + 1], np.r_[w[r][ids, h], 0.0] + ref.mass[:, 0], ref.reach)
            assert np.all(got[r, h, budget + 1:] == 0)
    assert s.pool.device_status() == 0


@pytest.mark.parametrize("n_docs,budget", [(9, 700), (40, 3000), (150, 40)])
def test_evict_long(L, n_docs, budget):
    s = Scenario(L, [([1000 - 7 * (j % 5) for j in range(n_docs)], 20, 0), ([30], 5, 0)], hq=2, hkv=2, seed=27, extra=2 * 200)
    check_evict(L, s, weights_of(s, "ties", np.random.default_rng(28)), budget, 4, 33)


@pytest.mark.parametrize("budget", [2**31 - 1, 2**31 - 5000])
def test_evict_with_the_largest_budgets(L, budget):
    """`kept` of 8 GB for a short cache: everything stays, the rest of it is -1."""
    s = Scenario(L, [([20], 9, 0)], hq=2, hkv=1, seed=49, extra=4)
    pages = s.pool.alloc_pages(3)
    dst = torch.from_numpy(L.pack_entries(pages, [0] * 3, [0] * 3, [1] * 3).view(np.int64).copy()).cuda()
    off = torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    kept = torch.full((1, 1, budget), -7, dtype=torch.int32, device="cuda")
    mass = torch.rand(s.n_entries(), 1, 16, device="cuda")
    L.lazyattn_evict(s.pool.handle, s.batch.c, mass, budget, 4, 8, dst, off, kept)
    assert s.pool.device_status() == 0
    assert torch.equal(kept[0, 0, :29].cpu(), torch.arange(29).int()) and bool((kept[0, 0, 29:] == -1).all())
    assert [oracle.unpack_entry(int(e))[2] for e in dst.cpu().numpy().view(np.uint64)] == [16, 13, 0]


@pytest.mark.parametrize("reserve", [0, 2])
def test_batch_evict_takes_no_more_pages_than_a_request_can_fill(L, reserve):
    """A budget past what the short requests hold, and a pool with pages for what they do hold: served, everything of them
    kept; a request without entries gets its reserve alone."""
    s = Scenario(L, [([400, 300], 30, 0), ([20], 9, 0), ([], 5, 0), ([], 0, 0)], seed=58, spare=0)
    w = [np.abs(x) for x in weights_of(s, "normal", np.random.default_rng(59))]
    mass = torch.from_numpy(s.mass_of(w).astype(np.float32)).cuda()
    n = [13 + reserve, 3 + reserve, 1 + reserve, reserve]                     # budget 200; 3, 1 and no entries
    s.pool.alloc_pages(s.pool.free_count() - sum(n))
    batch, kept, new = s.batch.evict(s.pool, mass, 200, sinks=4, recent=16, reserve=reserve)
    assert s.pool.free_count() == 0 and s.pool.device_status() == 0
    assert np.diff(batch.offsets_host).tolist() == n and batch.max_entries == n[0] and batch.c.n_entries == sum(n)
    got = [oracle.unpack_entry(int(e))[2] for e in batch.entries_host]
    assert got[:13] == [16] * 12 + [8] and got[n[0]:n[0] + 3] == [16, 13, 0] and got[n[0] + n[1]] == 5
    new, kept = new.cpu().numpy(), kept.cpu().numpy()
    for r in range(4):
        for h in range(s.hkv):
            ids = kept_tokens(w[r][:, h], 200, 4, 16) if len(w[r]) else []
            np.testing.assert_array_equal(kept[r, h], np.r_[s.pos[r][ids] if len(ids) else [], np.full(200 - len(ids), -1)])
            flat = new[batch.offsets_host[r]:batch.offsets_host[r + 1], h].reshape(-1)
            np.testing.assert_array_equal(flat, np.r_[w[r][ids, h] if len(ids) else [], np.zeros(len(flat) - len(ids))])


def test_batch_evict_of_nothing(L):
    s = Scenario(L, [([], 0, 0), ([], 0, 0)], seed=60, spare=0)
    mass = torch.zeros(1, s.hkv, 16, device="cuda")
    batch, kept, new = s.batch.evict(s.pool, mass, 32, reserve=0)
    assert s.pool.device_status() == 0 and bool((kept == -1).all())
    assert len(batch.entries_host) == 0 and batch.max_entries == 0 and batch.c.n_entries == 0


def test_evict_refuses_bad_tables_on_the_device(L):
    """Entries that go down in position, a page out of range, too few new entries, a new page out of range: that request
    keeps nothing and is reported; the other request is served."""
    for fault in ["order", "page", "few", "new page"]:
        s = Scenario(L, [([40, 30], 20, 0), ([50], 9, 0)], seed=29, extra=8)
        ent = s.batch.entries_host.copy()
        if fault == "order":
            ent[[0, 1]] = ent[[1, 0]]
        if fault == "page":
            ent[1] = (ent[1] & ~np.uint64(0xFFFFFFFF)) | np.uint64(s.pool.num_pages)
        b = s.batch.with_entries(ent, 0)
        pages = np.array(s.pool.alloc_pages(4))
        if fault == "new page":
            pages[1] = s.pool.num_pages + 5
        offs = [0, 1, 3] if fault == "few" else [0, 2, 4]
        dst = torch.from_numpy(L.pack_entries(pages, [0] * 4, [0] * 4, [1] * 4).view(np.int64).copy()).cuda()
        off = torch.tensor(offs, dtype=torch.int32, device="cuda")
        kept = torch.zeros(2, s.hkv, 20, dtype=torch.int32, device="cuda")
        mass = torch.ones(s.n_entries(), s.hkv, 16, device="cuda")
        dm = torch.full((4, s.hkv, 16), float("nan"), device="cuda")
        k0 = s.pool.k_pool.clone()
        L.lazyattn_evict(s.pool.handle, b.c, mass, 20, 1, 2, dst, off, kept, dm)
        assert s.pool.device_status() == L.LAZYATTN_ERANGE, fault
        kept, dst = kept.cpu().numpy(), dst.cpu().numpy().view(np.uint64)
        assert np.all(kept[0] == -1) and np.all(kept[1] >= 0)
        assert all(oracle.unpack_entry(int(e))[2] == 0 for e in dst[:offs[1]])
        assert sum(oracle.unpack_entry(int(e))[2] for e in dst[offs[1]:offs[2]]) == 20
        assert np.all(dm.cpu().numpy()[:offs[1]] == 0)
        touched = (s.pool.k_pool != k0).flatten(1).any(1).cpu().numpy().nonzero()[0]
        assert set(touched) <= set(pages[offs[1]:offs[2]])


# ------------------------------------------------------------------------------------------------ long tables

def with_empty_entries(L, s, lead, every):
    """The scenario's table with `lead` empty entries in front of each request's and `every` behind each of its entries."""
    b, out, offs = s.batch, [], [0]
    empty = L.pack_entries([0], [0], [0], [0])[0]
    for r in range(len(s.rows)):
        words = [empty] * lead
        for e in b.entries_host[b.offsets_host[r]:b.offsets_host[r + 1]]:
            words.append(e)
            if not oracle.unpack_entry(int(e))[3]:          # the writable run stays in one piece
                words += [empty] * every
        out += words
        offs.append(len(out))
    b2 = b.with_entries(np.array(out, np.uint64), b.flags)
    b2.offsets_host = np.array(offs, np.int32)
    b2.entry_offsets = torch.from_numpy(b2.offsets_host).cuda()
    b2.max_entries = int(np.max(np.diff(b2.offsets_host)))
    b2.c = L.lazyattn.make_batch(b2.num_requests, b2.max_entries, b2.entries, b2.entry_offsets, b.q_offsets, b.q_start,
                                 b.max_q_len, b.total_q, b.flags)
    s.batch = b2


@pytest.mark.parametrize("lead,every", [(70000, 0), (0, 900), (3, 2)])
def test_tables_of_many_entries(L, lead, every):
    """Tables past the prefill's 8192 marked tiles and past what an evicting block holds at a time, most entries empty."""
    s = Scenario(L, [([700, 33, 500], 40, 40), ([5, 100], 17, 9)], seed=34, extra=200)
    with_empty_entries(L, s, lead, every)
    check_prefill_window(L, s, 300, 3)
    check_prefill_mass(L, s, 1.0, False)
    check_evict(L, s, weights_of(s, "ties", np.random.default_rng(35)), 333, 4, 50)
    check_evict(L, s, weights_of(s, "equal", np.random.default_rng(36)), 1000, 0, 0)
    check_decode_window(L, s, 300, 3, 1)
    s = Scenario(L, [([700, 33, 500], 40, 0), ([5, 100], 17, 0)], seed=37)
    with_empty_entries(L, s, lead, every)
    check_decode_mass(L, s, 1.0, 2)


@pytest.mark.parametrize("a,b", [(0, 1), (3, 700), (700, 701), (1, 60000), (59000, 60000)])
def test_evict_finds_disorder_anywhere(L, a, b):
    """Two tokens' entries exchanged in a table that several blocks and segments share."""
    s = Scenario(L, [([], 16 * 60, 0), ([40], 5, 0)], seed=40, extra=12)
    with_empty_entries(L, s, 0, 0)
    words = list(s.batch.entries_host)
    empty = L.pack_entries([0], [0], [0], [0])[0]
    table = np.full(61000, empty, np.uint64)
    at = np.unique(np.r_[[0, 1, 3, 700, 701, 59000, 60000], np.linspace(5, 58000, 53).astype(int)])[:60]
    table[at] = words[:len(at)]
    fine = table.copy()
    table[[a, b]] = table[[b, a]]
    for ent, bad in [(fine, False), (table, True)]:
        e = torch.from_numpy(ent.view(np.int64).copy()).cuda()
        off = torch.tensor([0, len(ent)], dtype=torch.int32, device="cuda")
        c = L.lazyattn.make_batch(1, len(ent), e, off)
        dst = torch.from_numpy(L.pack_entries(s.pool.alloc_pages(4), [0] * 4, [0] * 4, [1] * 4).view(np.int64).copy()).cuda()
        d_off = torch.tensor([0, 4], dtype=torch.int32, device="cuda")
        kept = torch.zeros(1, s.hkv, 50, dtype=torch.int32, device="cuda")
        mass = torch.rand(len(ent), s.hkv, 16, device="cuda")
        L.lazyattn_evict(s.pool.handle, c, mass, 50, 4, 8, dst, d_off, kept)
        assert (s.pool.device_status() == L.LAZYATTN_ERANGE) == bad
        assert bool((kept == -1).all()) == bad and bool((kept >= 0).all()) != bad


def test_calls_on_a_stream_of_their_own(L):
    """stream= given: the calls run there, behind work that fills their inputs, with another stream current."""
    s = Scenario(L, [([300, 150], 64, 64)], seed=38, extra=40)
    side = torch.cuda.Stream()
    q, want = s.dev(s.q), s.empty(64, s.hq, s.d)
    wsp, wsm = workspace(L, s, L.LAZYATTN_OP_PREFILL, 100, 4), workspace(L, s, L.LAZYATTN_OP_PREFILL_MASS)
    L.lazyattn_prefill_window(s.pool.handle, s.batch.c, q, want, 100, 4, *wsp)
    mass = torch.empty(s.n_entries(), s.hkv, 16, device="cuda")
    L.lazyattn_prefill_mass(s.pool.handle, s.batch.c, q, None, mass, 1.0, *wsm)
    batch, kept, _ = s.batch.evict(s.pool, mass, 50, 2, 8)
    torch.cuda.synchronize()
    late, out, mass2 = torch.zeros_like(q), torch.zeros_like(want), torch.empty_like(mass)
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        late.copy_(q)
    L.lazyattn_prefill_window(s.pool.handle, s.batch.c, late, out, 100, 4, *wsp, stream=side)
    L.lazyattn_prefill_mass(s.pool.handle, s.batch.c, late, None, mass2, 1.0, *wsm, stream=side)
    batch2, kept2, _ = s.batch.evict(s.pool, mass2, 50, 2, 8, stream=side)
    side.synchronize()
    assert torch.equal(out, want) and torch.equal(mass, mass2) and torch.equal(kept, kept2)


def test_two_calls_at_once(L):
    """Two pools' calls in flight on two streams, each with a workspace of its own: the bits of the calls one by one."""
    both = [Scenario(L, [([900, 150], 130, 130), ([33], 20, 20)], seed=56, extra=400),
            Scenario(L, [([400] * 6, 64, 64)], seed=57, hq=8, hkv=1, extra=400)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    work = []
    for s in both:
        R = len(s.rows)
        st = dict(q=s.dev(s.q), step=[s.dev(x) for x in step_inputs(s, R)], table=s.batch.entries.clone(), R=R,
                  wsp=workspace(L, s, L.LAZYATTN_OP_PREFILL, 700, 4), wsw=workspace(L, s, L.LAZYATTN_OP_DECODE, 700, 4),
                  wsm=workspace(L, s, L.LAZYATTN_OP_PREFILL_MASS), wsd=workspace(L, s, L.LAZYATTN_OP_DECODE_MASS),
                  off=torch.arange(R + 1, dtype=torch.int32, device="cuda") * 20,
                  pages=torch.from_numpy(L.pack_entries(s.pool.alloc_pages(20 * R), [0] * 20 * R, [0] * 20 * R, [1] * 20 * R)
                                         .view(np.int64).copy()).cuda())
        work.append(st)

    def outputs(s, st):
        rows, R = s.batch.total_q, st["R"]
        return dict(p=s.empty(rows, s.hq, s.d), w=s.empty(R, s.hq, s.d), d=s.empty(R, s.hq, s.d), dst=st["pages"].clone(),
                    m=torch.zeros(s.n_entries(), s.hkv, 16, device="cuda"), n=torch.zeros(s.n_entries(), s.hkv, 16, device="cuda"),
                    kept=torch.zeros(R, s.hkv, 300, dtype=torch.int32, device="cuda"))

    def calls(s, st, o):
        h, c, (q1, k1, v1) = s.pool.handle, s.batch.c, st["step"]
        L.lazyattn_prefill_window(h, c, st["q"], o["p"], 700, 4, *st["wsp"])
        L.lazyattn_prefill_mass(h, c, st["q"], None, o["m"], 1.0, *st["wsm"])
        s.batch.entries.copy_(st["table"])
        L.lazyattn_decode_window(h, c, q1, k1, v1, o["w"], 700, 4, *st["wsw"])
        s.batch.entries.copy_(st["table"])
        L.lazyattn_decode_mass(h, c, q1, k1, v1, o["d"], o["m"], o["n"], 0.5, *st["wsd"])
        L.lazyattn_evict(h, c, o["n"], 300, 4, 16, o["dst"], st["off"], o["kept"])

    want = []
    for s, st in zip(both, work):
        o = outputs(s, st)
        calls(s, st, o)
        torch.cuda.synchronize()
        want.append(o)
    got = [[outputs(s, st) for _ in range(10)] for s, st in zip(both, work)]
    torch.cuda.synchronize()
    for i in range(10):
        for j in (0, 1):
            with torch.cuda.stream(streams[j]):
                calls(both[j], work[j], got[j][i])
    torch.cuda.synchronize()
    for j in (0, 1):
        for o in got[j]:
            for name, x in o.items():
                assert torch.equal(x, want[j][name]), (j, name)
        assert both[j].pool.device_status() == 0


# ------------------------------------------------------------------------------------------------ long tables, every layout

@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("hq,hkv,window", [(8, 2, 3000), (8, 1, 2300), (2, 2, 4000)])
def test_prefill_window_split_modes(L, mode, hq, hkv, window):
    """Windows of so many tiles that several blocks share them, in every layout: ragged documents, rows of one block and
    of two, a request whose window is all it has."""
    s = Scenario(L, [([900, 77, 900, 1000, 1000], 70, 70), ([500, 1000, 1000, 33], 21, 9), ([], 60, 60)], mode, hq=hq, hkv=hkv,
                 seed=50)
    assert workspace(L, s, L.LAZYATTN_OP_PREFILL, window, 20)[1] > 256       # room for partials: the call splits
    check_prefill_window(L, s, window, 20)


@pytest.mark.parametrize("mode", MODES)
def test_long_modes(L, mode):
    """The other calls over tables that several blocks share, in every layout."""
    s = Scenario(L, [([900, 77, 900, 1000], 130, 130), ([500, 1000, 33], 21, 9)], mode, hq=8, hkv=2, seed=51)
    check_prefill_mass(L, s, 1.0, True)
    for check in (lambda s: check_decode_window(L, s, 2000, 20, 2), lambda s: check_decode_mass(L, s, 0.5, 2)):
        check(Scenario(L, [([900, 77, 900, 1000], 130, 0), ([500, 1000, 33], 21, 0)], mode, hq=8, hkv=2, seed=52))


# ------------------------------------------------------------------------------------------------ a wrong bound

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("op", ["evict", "decode_mass", "prefill_mass"])
def test_more_entries_than_the_batch_says(L, op, dtype):
    """max_entries below a request's entries: reported; eviction keeps nothing of it, mass and output take the first
    max_entries entries and leave the others' mass alone; the request within the bound is served."""
    s = Scenario(L, [([100], 30, 8), ([20], 9, 4)], dtype=dtype, hq=4, hkv=2, seed=45, extra=12)
    b, cap = s.batch, 6                                                       # the requests have 10 and 4 entries
    b.c = L.lazyattn.make_batch(2, cap, b.entries, b.entry_offsets, b.q_offsets, b.q_start, b.max_q_len, b.total_q)
    if op == "evict":
        pages = s.pool.alloc_pages(12)
        dst = torch.from_numpy(L.pack_entries(pages, [0] * 12, [0] * 12, [1] * 12).view(np.int64).copy()).cuda()
        off = torch.tensor([0, 10, 12], dtype=torch.int32, device="cuda")
        kept = torch.full((2, s.hkv, 125), -7, dtype=torch.int32, device="cuda")
        mass = torch.full((s.n_entries(), s.hkv, 16), 0.5, device="cuda")
        dm = torch.full((12, s.hkv, 16), float("nan"), device="cuda")
        k0 = s.pool.k_pool.clone()
        L.lazyattn_evict(s.pool.handle, b.c, mass, 125, 0, 0, dst, off, kept, dm)
        assert s.pool.device_status() == L.LAZYATTN_ERANGE
        assert [oracle.unpack_entry(int(e))[2] for e in dst.cpu().numpy().view(np.uint64)] == [0] * 10 + [16, 13]
        assert bool((kept[0] == -1).all()) and bool((dm[:10] == 0).all())
        assert torch.equal(kept[1].cpu(), torch.cat([torch.arange(29), torch.full((96,), -1)]).int().expand(s.hkv, 125))
        touched = (s.pool.k_pool != k0).flatten(1).any(1).cpu().numpy().nonzero()[0]
        assert set(touched) == set(pages[10:])
        return
    got = torch.full((s.n_entries(), s.hkv, 16), float("nan"), device="cuda")
    take = [16 * cap, 29]                                                     # tokens of the entries that take part
    if op == "decode_mass":
        ws, n = workspace(L, s, L.LAZYATTN_OP_DECODE_MASS)
        q, kn, vn = step_inputs(s, 2)
        out = s.empty(2, s.hq, s.d)
        L.lazyattn_decode_mass(s.pool.handle, b.c, s.dev(q), s.dev(kn), s.dev(vn), out, None, got, 1.0, ws, n)
        ks = [s.k[0][:96], np.r_[s.k[1], kn[1][None]]]
        vs = [s.v[0][:96], np.r_[s.v[1], vn[1][None]]]
        refs = [attend(s.spec, q[r][None], ks[r], vs[r], [130 if r == 0 else 29], np.arange(len(ks[r]))) for r in range(2)]
        for r in range(2):
            check_out(out.float().cpu().numpy()[r], refs[r], dtype, row=0)
    else:
        ws, n = workspace(L, s, L.LAZYATTN_OP_PREFILL_MASS)
        L.lazyattn_prefill_mass(s.pool.handle, b.c, s.dev(s.q), None, got, 1.0, ws, n)
        refs = [attend(s.spec, s.q[s.row_slice(r)], s.k[r][:take[r]], s.v[r][:take[r]], s.starts[r] + np.arange(s.rows[r]),
                       np.arange(take[r])) for r in range(2)]
    assert s.pool.device_status() == L.LAZYATTN_ERANGE
    got = got.cpu().numpy()
    assert np.all(np.isnan(got[cap:10]))
    got[cap:10] = 0
    pad = [np.r_[refs[0].mass, np.zeros((34 + (op == "decode_mass"), s.hkv))], refs[1].mass]
    check_mass(got, s.mass_of(pad), max(x.reach for x in refs))


@pytest.mark.parametrize("op", ["prefill", "prefill_window"])
def test_split_rows_past_total_q(L, op):
    """A request whose rows end past total_q, in a call that splits the keys over several blocks: reported, and nothing is
    written for it, neither its rows inside total_q nor what lies behind."""
    s = Scenario(L, [([900] * 4, 20, 20), ([500], 30, 30)], seed=48)
    b, top = s.batch, 40                                                      # rows 0..19, 20..49; total_q 40
    c = L.lazyattn.make_batch(2, b.max_entries, b.entries, b.entry_offsets, b.q_offsets, b.q_start, b.max_q_len, top)
    out = s.empty(64, s.hq, s.d)
    if op == "prefill":
        n = L.lazyattn_workspace_size(s.pool.handle, L.LAZYATTN_OP_PREFILL, c)
    else:
        n = L.lazyattn_window_workspace_size(s.pool.handle, L.LAZYATTN_OP_PREFILL, c, 3000, 4)
    assert n > 256                                                            # room for partials: the call splits
    ws = torch.zeros(n, dtype=torch.uint8, device="cuda")
    q = s.dev(s.q)
    if op == "prefill":
        L.lazyattn_prefill(s.pool.handle, c, q, out, ws, n)
    else:
        L.lazyattn_prefill_window(s.pool.handle, c, q, out, 3000, 4, ws, n)
    assert s.pool.device_status() == L.LAZYATTN_ERANGE
    got = out.float().cpu().numpy()
    assert np.all(np.isnan(got[20:]))
    want = attend(s.spec, s.q[:20], s.k[0], s.v[0], s.starts[0] + np.arange(20), s.pos[0], 3000 if op != "prefill" else None, 4)
    check_out(got[:20], want, "bf16")


# ------------------------------------------------------------------------------------------------ refusals

def test_refusals(L):
    s = Scenario(L, [([40, 30], 20, 8)], seed=30, extra=4)
    q, out = s.dev(s.q), s.empty(8, s.hq, s.d)
    q1, k1, v1 = (s.dev(x) for x in step_inputs(s, 1))
    o1 = s.empty(1, s.hq, s.d)
    mass = torch.zeros(s.n_entries(), s.hkv, 16, device="cuda")
    dst = torch.from_numpy(L.pack_entries(s.pool.alloc_pages(2), [0] * 2, [0] * 2, [1] * 2).view(np.int64).copy()).cuda()
    off = torch.tensor([0, 2], dtype=torch.int32, device="cuda")
    kept = torch.full((1, s.hkv, 20), -7, dtype=torch.int32, device="cuda")
    h, c = s.pool.handle, s.batch.c
    wsw, nw = workspace(L, s, L.LAZYATTN_OP_DECODE, 8, 0)
    wsp, npm = workspace(L, s, L.LAZYATTN_OP_PREFILL_MASS)
    wsd, ndm = workspace(L, s, L.LAZYATTN_OP_DECODE_MASS)
    EINVAL, EWS = L.LAZYATTN_EINVAL, L.LAZYATTN_EWORKSPACE
    odd = torch.zeros(4 * mass.numel(), device="cuda")[1:1 + mass.numel()]
    nan = float("nan")
    calls = [
        (EINVAL, lambda: L.lazyattn_prefill_window(h, c, q, out, 0, 0)),
        (EINVAL, lambda: L.lazyattn_prefill_window(h, c, q, out, -5, 0)),
        (EINVAL, lambda: L.lazyattn_prefill_window(h, c, q, out, 8, -1)),
        (EINVAL, lambda: L.lazyattn_prefill_window(h, c, None, out, 8, 0)),
        (EINVAL, lambda: L.lazyattn_prefill_window(h, c, q, None, 8, 0)),
        (EINVAL, lambda: L.lazyattn_prefill_window(h, c, q[:, :, ::2], out, 8, 0)),
        (EINVAL, lambda: L.lazyattn_decode_window(h, c, q1, k1, v1, o1, 0, 0, wsw, nw)),
        (EINVAL, lambda: L.lazyattn_decode_window(h, c, q1, None, v1, o1, 8, 0, wsw, nw)),
        (EINVAL, lambda: L.lazyattn_decode_window(h, c, q1, k1, v1, o1, 8, 0, None, nw)),
        (EINVAL, lambda: L.lazyattn_decode_window(h, c, q1, k1, v1, o1, 8, 0, wsw.data_ptr() + 16, nw)),
        (EWS, lambda: L.lazyattn_decode_window(h, c, q1, k1, v1, o1, 8, 0, wsw, nw - 1)),
        (EINVAL, lambda: L.lazyattn_prefill_mass(h, c, q, mass, mass, 1.5, wsp, npm)),
        (EINVAL, lambda: L.lazyattn_prefill_mass(h, c, q, mass, mass, -0.1, wsp, npm)),
        (EINVAL, lambda: L.lazyattn_prefill_mass(h, c, q, mass, mass, nan, wsp, npm)),
        (EINVAL, lambda: L.lazyattn_prefill_mass(h, c, q, mass, None, 1.0, wsp, npm)),
        (EINVAL, lambda: L.lazyattn_prefill_mass(h, c, None, mass, mass, 1.0, wsp, npm)),
        (EINVAL, lambda: L.lazyattn_prefill_mass(h, c, q, odd, mass, 1.0, wsp, npm)),
        (EINVAL, lambda: L.lazyattn_prefill_mass(h, c, q, mass.double(), mass, 1.0, wsp, npm)),
        (EWS, lambda: L.lazyattn_prefill_mass(h, c, q, mass, mass, 1.0, wsp, npm - 1)),
        (EINVAL, lambda: L.lazyattn_decode_mass(h, c, q1, k1, v1, o1, mass, mass, nan, wsd, ndm)),
        (EINVAL, lambda: L.lazyattn_decode_mass(h, c, q1, k1, v1, None, mass, mass, 1.0, wsd, ndm)),
        (EWS, lambda: L.lazyattn_decode_mass(h, c, q1, k1, v1, o1, mass, mass, 1.0, wsd, ndm - 1)),
        (EINVAL, lambda: L.lazyattn_evict(h, c, mass, 0, 0, 0, dst, off, kept)),
        (EINVAL, lambda: L.lazyattn_evict(h, c, mass, 20, -1, 0, dst, off, kept)),
        (EINVAL, lambda: L.lazyattn_evict(h, c, mass, 20, 11, 10, dst, off, kept)),
        (EINVAL, lambda: L.lazyattn_evict(h, c, mass, 20, 2**31 - 1, 2**31 - 1, dst, off, kept)),
        (EINVAL, lambda: L.lazyattn_evict(h, c, None, 20, 1, 1, dst, off, kept)),
        (EINVAL, lambda: L.lazyattn_evict(h, c, mass, 20, 1, 1, dst, off.long(), kept)),
        (EINVAL, lambda: L.lazyattn_evict(h, c, mass, 20, 1, 1, None, off, kept)),
        (EINVAL, lambda: L.lazyattn_evict(h, c, mass, 20, 1, 1, dst, off, None)),
    ]
    table = s.batch.entries.clone()
    for i, (code, call) in enumerate(calls):
        with pytest.raises(L.LazyAttnError) as e:
            call()
        assert e.value.code == code, i
    torch.cuda.synchronize()
    assert torch.equal(table, s.batch.entries) and bool((kept == -7).all()) and bool(torch.isnan(out).all())
    assert L.lazyattn_window_workspace_size(h, L.LAZYATTN_OP_DECODE, c, 0, 0) == 0
    assert L.lazyattn_window_workspace_size(h, L.LAZYATTN_OP_PREFILL_MASS, c, 8, 0) == 0


@pytest.mark.parametrize("mode", ["doc_local", "prerotated"])
def test_evict_refuses_keys_turned_to_their_place(L, mode):
    s = Scenario(L, [([40, 30], 20, 0)], mode, seed=31, extra=4)
    z = torch.zeros(64, dtype=torch.int64, device="cuda")
    with pytest.raises(L.LazyAttnError) as e:
        L.lazyattn_evict(s.pool.handle, s.batch.c, z.float(), 20, 1, 1, z, z.int(), z.int())
    assert e.value.code == L.LAZYATTN_EINVAL


# ------------------------------------------------------------------------------------------------ together

def test_a_cache_kept_small(L):
    """A prompt under a window, its last rows observing the cache, the cache cut down, decode steps that go on
    observing, a second cut, and a windowed step: each step against the 64-bit definition on the tokens then held."""
    s = Scenario(L, [([300, 150], 64, 64), ([200, 77, 130], 40, 40)], seed=32, hq=8, hkv=2, extra=200)
    R, hkv = 2, s.hkv
    check_prefill_window(L, s, 128, 4)
    ws, n = workspace(L, s, L.LAZYATTN_OP_PREFILL_MASS)
    mass = torch.empty(s.n_entries(), hkv, 16, device="cuda")
    L.lazyattn_prefill_mass(s.pool.handle, s.batch.c, s.dev(s.q), None, mass, 1.0, ws, n)
    # per request and head: the tokens held, in order
    held = [[(s.k[r][:, h], s.v[r][:, h]) for h in range(hkv)] for r in range(R)]
    batch, free0 = s.batch, s.pool.free_count()
    for budget, steps in [(128, 5), (64, 3)]:
        m = mass.cpu().numpy()
        weights = [np.concatenate([m[i, :, :oracle.unpack_entry(int(e))[2]].T for i, e in
                                   zip(range(batch.offsets_host[r], batch.offsets_host[r + 1]),
                                       batch.entries.cpu().numpy().view(np.uint64)[batch.offsets_host[r]:])]) for r in range(R)]
        batch, kept, mass = batch.evict(s.pool, mass, budget, sinks=4, recent=16, reserve=1)
        for r in range(R):
            for h in range(hkv):
                ids = kept_tokens(weights[r][:, h], budget, 4, 16)
                held[r][h] = (held[r][h][0][ids], held[r][h][1][ids])
        wsd_n = L.lazyattn_workspace_size(s.pool.handle, L.LAZYATTN_OP_DECODE_MASS, batch.c)
        wsd = torch.zeros(wsd_n, dtype=torch.uint8, device="cuda")
        for t in range(steps):
            q, kn, vn = step_inputs(s, R)
            out = s.empty(R, s.hq, s.d)
            old = mass.clone()
            L.lazyattn_decode_mass(s.pool.handle, batch.c, s.dev(q), s.dev(kn), s.dev(vn), out, mass, mass, 1.0, wsd, wsd_n)
            got, add = out.float().cpu().numpy(), (mass - old).cpu().numpy()
            for r in range(R):
                for h in range(hkv):
                    k, v = held[r][h]
                    held[r][h] = np.r_[k, kn[r, h][None]], np.r_[v, vn[r, h][None]]
                    k, v = held[r][h]
                    g = s.hq // hkv
                    want = attend(s.spec, q[r, h * g:(h + 1) * g][None], k[:, None], v[:, None], [len(k) - 1],
                                            np.arange(len(k)))
                    check_out(got[r, h * g:(h + 1) * g], want, "bf16", row=0)
                    e0 = batch.offsets_host[r]
                    seen = add[e0:batch.offsets_host[r + 1], h].reshape(-1)
                    # the difference of two float32 totals below 256: half a step of each
                    assert np.max(np.abs(seen[:len(k)] - want.mass[:, 0])) <= 2.0 ** -16 + want.reach * 1e-5
                    assert np.all(seen[len(k):] == 0)
    wn = L.lazyattn_window_workspace_size(s.pool.handle, L.LAZYATTN_OP_DECODE, batch.c, 20, 4)
    wsw = torch.zeros(wn, dtype=torch.uint8, device="cuda")
    q, kn, vn = step_inputs(s, R)
    out = s.empty(R, s.hq, s.d)
    L.lazyattn_decode_window(s.pool.handle, batch.c, s.dev(q), s.dev(kn), s.dev(vn), out, 20, 4, wsw, wn)
    got = out.float().cpu().numpy()
    for r in range(R):
        k = np.stack([np.r_[held[r][h][0], kn[r, h][None]] for h in range(hkv)], 1)
        v = np.stack([np.r_[held[r][h][1], vn[r, h][None]] for h in range(hkv)], 1)
        want = attend(s.spec, q[r][None], k, v, [len(k) - 1], np.arange(len(k)), 20, 4)
        check_out(got[r], want, "bf16", row=0)
    assert s.pool.device_status() == 0
    assert s.pool.free_count() < free0


def test_captured_and_replayed(L):
    """Every call in one CUDA graph on a side stream, replayed: the same bits as the eager calls."""
    s = Scenario(L, [([300, 150], 64, 64), ([200, 77, 130], 40, 40)], seed=33, extra=64)
    R = 2
    q1, k1, v1 = (s.dev(x) for x in step_inputs(s, R))
    q = s.dev(s.q)
    per = 6
    dst0 = torch.from_numpy(L.pack_entries(s.pool.alloc_pages(R * per), [0] * R * per, [0] * R * per, [1] * R * per)
                            .view(np.int64).copy()).cuda()
    off = torch.arange(R + 1, dtype=torch.int32, device="cuda") * per
    entries0 = s.batch.entries.clone()
    wsp = workspace(L, s, L.LAZYATTN_OP_PREFILL, 100, 4)
    wsw = workspace(L, s, L.LAZYATTN_OP_DECODE, 100, 4)
    wsm = workspace(L, s, L.LAZYATTN_OP_PREFILL_MASS)
    wsd = workspace(L, s, L.LAZYATTN_OP_DECODE_MASS)
    o = [s.empty(s.batch.total_q, s.hq, s.d), s.empty(R, s.hq, s.d), s.empty(R, s.hq, s.d)]
    m = [torch.empty(s.n_entries(), s.hkv, 16, device="cuda") for _ in range(2)]
    dst, kept, dm = dst0.clone(), torch.zeros(R, s.hkv, 80, dtype=torch.int32, device="cuda"), torch.empty(R * per, s.hkv, 16, device="cuda")

    def calls():
        h, c = s.pool.handle, s.batch.c
        s.batch.entries.copy_(entries0)
        L.lazyattn_prefill_window(h, c, q, o[0], 100, 4, *wsp)
        L.lazyattn_prefill_mass(h, c, q, None, m[0], 1.0, *wsm)
        L.lazyattn_decode_window(h, c, q1, k1, v1, o[1], 100, 4, *wsw)
        L.lazyattn_decode_mass(h, c, q1, k1, v1, o[2], m[0], m[1], 0.5, *wsd)
        L.lazyattn_evict(h, c, m[1], 80, 4, 16, dst, off, kept, dm)

    results = o + m + [dst, kept, dm]
    calls()
    torch.cuda.synchronize()
    want = [x.clone() for x in results]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        calls()
    for _ in range(3):
        for x in results[:-3] + [kept, dm]:
            x.zero_()
        dst.copy_(dst0)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(results, want):
            assert torch.equal(a, b)
    assert s.pool.device_status() == 0


@pytest.mark.parametrize("op", ["decode", "decode_window", "decode_mass"])
def test_a_table_written_just_before_a_step(L, op):
    """A kernel that rewrites the table runs directly before the step, with nothing waited for in between: the step
    reads the new table, whichever way its own launches overlap."""
    s = Scenario(L, [([160, 320], 10, 0), ([480], 21, 0)], seed=39)
    R = 2
    q, k, v = (s.dev(x) for x in step_inputs(s, R))
    first = s.batch.entries.clone()
    host = first.cpu().numpy().view(np.uint64).copy()
    off = s.batch.offsets_host
    low = np.uint64(0xFFFFFFFF)
    for r in range(R):   # the document pages in the opposite order
        i = np.arange(off[r], off[r] + 30)
        host[i] = (host[i] & ~low) | (host[i[::-1]] & low)
    second = torch.from_numpy(host.view(np.int64).copy()).cuda()
    code = {"decode": L.LAZYATTN_OP_DECODE, "decode_mass": L.LAZYATTN_OP_DECODE_MASS}.get(op)
    ws, n = workspace(L, s, code) if code is not None else workspace(L, s, L.LAZYATTN_OP_DECODE, 200, 4)
    mass = torch.zeros(s.n_entries(), s.hkv, 16, device="cuda")

    def step(table, wait):
        out = s.empty(R, s.hq, s.d)
        torch.add(table, 0, out=s.batch.entries)
        if wait:
            torch.cuda.synchronize()
        if op == "decode":
            L.lazyattn_decode(s.pool.handle, s.batch.c, q, k, v, out, ws, n)
        elif op == "decode_window":
            L.lazyattn_decode_window(s.pool.handle, s.batch.c, q, k, v, out, 200, 4, ws, n)
        else:
            L.lazyattn_decode_mass(s.pool.handle, s.batch.c, q, k, v, out, None, mass, 1.0, ws, n)
        return out

    want = [step(first, True), step(second, True)]
    torch.cuda.synchronize()
    assert not torch.equal(*want)
    got = [step((first, second)[i % 2], False) for i in range(40)]
    for i, x in enumerate(got):
        assert torch.equal(x, want[i % 2])
    assert s.pool.device_status() == 0
