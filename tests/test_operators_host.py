"""Rotary positions, tree attention and reading back: what needs no GPU -- the
frequency schedules, and the refusals of bad calls (on a cache over a host
buffer that nothing dereferences)."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

from test_abi_host import _host_cache

INVALID, STATE, WORKSPACE = 1, 3, 6


@pytest.fixture(scope="module")
def kvq():
    from mixed_precision_kv_kvq_b200 import build

    build.build()
    import mixed_precision_kv_kvq_b200 as m

    m.load()
    return m


# ------------------------------------------------------------- frequencies

@pytest.mark.parametrize("d", [2, 6, 64, 96, 128])
@pytest.mark.parametrize("theta", [10000.0, 500000.0])
def test_freqs_plain_linear_ntk(kvq, d, theta):
    want = np.array([theta ** (-2.0 * p / d) for p in range(d // 2)])
    inv, mag = kvq.kvq_rope_freqs(d, theta)
    assert mag == 1.0 and np.allclose(inv, want, rtol=1e-14, atol=0)
    inv, mag = kvq.kvq_rope_freqs(d, theta, kvq.KVQ_ROPE_LINEAR, 4.0)
    assert mag == 1.0 and np.allclose(inv, want / 4.0, rtol=1e-14, atol=0)
    if d > 2:
        inv, _ = kvq.kvq_rope_freqs(d, theta, kvq.KVQ_ROPE_NTK, 4.0)
        base = theta * 4.0 ** (d / (d - 2))
        assert np.allclose(inv, [base ** (-2.0 * p / d) for p in range(d // 2)], rtol=1e-13, atol=0)
        # the fastest pair keeps its speed, the slowest is interpolated by the factor
        assert inv[0] == 1.0 and math.isclose(inv[-1], want[-1] / 4.0, rel_tol=1e-12)


def test_freqs_yarn(kvq):
    d, theta, s, orig = 128, 10000.0, 16.0, 4096
    inv, mag = kvq.kvq_rope_freqs(d, theta, kvq.KVQ_ROPE_YARN, s, orig)
    plain, _ = kvq.kvq_rope_freqs(d, theta)
    assert math.isclose(mag, 0.1 * math.log(16.0) + 1.0, rel_tol=2 ** -23)
    turns = plain * orig / (2 * math.pi)
    ratio = inv / plain
    assert np.all(np.diff(ratio) <= 1e-12)  # from unchanged to interpolated
    assert np.allclose(ratio[turns > 40], 1.0) and np.allclose(ratio[turns < 0.8], 1 / s)
    mid = (turns > 1.3) & (turns < 25)
    assert np.all(ratio[mid] < 1.0) and np.all(ratio[mid] > 1 / s)
    # factor 1 changes nothing
    inv, mag = kvq.kvq_rope_freqs(d, theta, kvq.KVQ_ROPE_YARN, 1.0, orig)
    assert mag == 1.0 and np.allclose(inv, plain, rtol=1e-15)


@pytest.mark.parametrize("args", [
    (0, 1e4, 0, 1.0, 0), (3, 1e4, 0, 1.0, 0), (130, 1e4, 0, 1.0, 0),   # rot_dim
    (64, 1.0, 0, 1.0, 0), (64, float("nan"), 0, 1.0, 0),               # theta
    (64, 1e4, 4, 1.0, 0), (64, 1e4, -1, 1.0, 0),                       # scaling
    (64, 1e4, 1, 0.5, 0), (64, 1e4, 2, float("inf"), 0),               # factor
    (2, 1e4, 2, 2.0, 0), (64, 1e4, 3, 2.0, 0),                         # NTK on one pair; YaRN without a length
])
def test_freqs_refusals(kvq, args):
    with pytest.raises(kvq.KVQError) as e:
        kvq.kvq_rope_freqs(*args)
    assert e.value.status == INVALID


def test_rope_schedule_object(kvq):
    r = kvq.Rope(64, layout="interleaved", inv_freq=np.ones(32), magnitude=2.0)
    assert r.magnitude == 2.0 and r.inv_freq.tolist() == [1.0] * 32
    for bad in (dict(layout="pairs"), dict(scaling="dynamic"), dict(rot_dim=64, inv_freq=np.ones(31))):
        with pytest.raises(ValueError):
            kvq.Rope(**bad)


# ---------------------------------------------------------------- refusals

class Rows(C.Structure):
    """kvq_rows of include/kvq.h."""
    _fields_ = [("data", C.c_void_p), ("stride_b", C.c_longlong), ("stride_t", C.c_longlong), ("stride_h", C.c_longlong)]


def _rows(kvq, ptr, b=512, t=256, h=128):
    return Rows(ptr, b, t, h)


def _rope(kvq, **kw):
    """kvq_rope with good arguments but for those given; -> status.  Never launches: every call here is refused."""
    buf = np.zeros(4096, np.uint8)
    base = buf.ctypes.data + (-buf.ctypes.data) % 16
    a = dict(rot_dim=128, layout=0, inv=np.ones(64), mag=1.0, pos=base, pos_type=1, batch=1, n=1, dtype=0,
             q=_rows(kvq, base), q_out=_rows(kvq, base), q_heads=2, k=None, k_out=None, kv_heads=0)
    a.update(kw)
    ref = lambda x: C.byref(x) if x is not None else None  # noqa: E731
    inv = a["inv"].ctypes.data_as(C.c_void_p) if a["inv"] is not None else None
    return kvq.load().kvq_rope(a["rot_dim"], a["layout"], inv, a["mag"], a["pos"], a["pos_type"], 1, 1, a["batch"], a["n"],
                               a["dtype"], ref(a["q"]), ref(a["q_out"]), a["q_heads"], ref(a["k"]), ref(a["k_out"]),
                               a["kv_heads"], None)


@pytest.mark.parametrize("bad", [
    dict(rot_dim=0), dict(rot_dim=127), dict(rot_dim=130), dict(layout=2), dict(pos_type=2), dict(dtype=2), dict(inv=None),
    dict(inv=np.full(64, np.nan)), dict(inv=np.full(64, 2.0 ** 21)), dict(mag=float("inf")), dict(batch=-1), dict(n=-1),
    dict(q_heads=-1), dict(pos=None), dict(pos=4), dict(q=None), dict(q_out=None), dict(kv_heads=2),
], ids=lambda d: next(iter(d)))
def test_rope_refusals(kvq, bad):
    assert _rope(kvq, **bad) == INVALID
    assert kvq.kvq_last_error()


def test_rope_refuses_rows_off_their_elements(kvq):
    buf = np.zeros(4096, np.uint8)
    base = buf.ctypes.data + (-buf.ctypes.data) % 16
    assert _rope(kvq, q=_rows(kvq, base + 1)) == INVALID                       # half an element
    assert _rope(kvq, q=_rows(kvq, base + 2), layout=1) == INVALID             # half a pair
    assert _rope(kvq, q=_rows(kvq, base, h=129), layout=1) == INVALID
    assert _rope(kvq, q=_rows(kvq, base + 4), dtype=1, layout=1) == INVALID


def test_rope_of_nothing(kvq):
    assert _rope(kvq, batch=0) == 0 and _rope(kvq, n=0, pos=None) == 0 and _rope(kvq, q_heads=0, q=None, q_out=None) == 0


def _tree(kvq, h, pool, **kw):
    p = pool.ptr.value
    a = dict(layer=0, q=_rows(kvq, p), q_heads=4, n=3, k=_rows(kvq, p), v=_rows(kvq, p), dtype=0, mask=None, mask_b=0,
             scale=0.1, out=p, ws=p, ws_bytes=1 << 40)
    a.update(kw)
    ref = lambda x: C.byref(x) if x is not None else None  # noqa: E731
    return kvq.load().kvq_tree_attn(h, a["layer"], ref(a["q"]), a["q_heads"], a["n"], ref(a["k"]), ref(a["v"]), a["dtype"],
                                    a["mask"], a["mask_b"], a["scale"], a["out"], a["ws"], a["ws_bytes"], None)


def test_tree_refusals(kvq):
    h, pool = _host_cache(kvq)
    p = pool.ptr.value
    try:
        bad = [dict(layer=1), dict(layer=-1), dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(dtype=2),
               dict(q_heads=3), dict(q_heads=0), dict(q_heads=18), dict(n=0), dict(n=1025), dict(scale=float("nan")),
               dict(mask_b=-1), dict(out=p + 8), dict(q=_rows(kvq, p + 8)), dict(k=_rows(kvq, p, t=132)),
               dict(v=_rows(kvq, p, h=4)), dict(q=_rows(kvq, None))]
        for kw in bad:
            assert _tree(kvq, h, pool, **kw) == INVALID, kw
        for kw in (dict(ws=None), dict(ws_bytes=0), dict(ws=p + 4)):
            assert _tree(kvq, h, pool, **kw) == WORKSPACE, kw
        assert kvq.kvq_tree_workspace(h, 0, 4, 3) > 0
        for args in ((1, 4, 3), (0, 3, 3), (0, 18, 3), (0, 4, 0), (0, 4, 1025)):
            assert kvq.kvq_tree_workspace(h, *args) == 0
        assert kvq.load().kvq_tree_workspace(None, 0, 4, 3) == 0
    finally:
        kvq.kvq_free(h)


def test_read_refusals(kvq):
    h, pool = _host_cache(kvq)
    p = pool.ptr.value
    lib = kvq.load()
    rows = lambda *a, **k: C.byref(_rows(kvq, *a, **k))  # noqa: E731
    try:
        assert lib.kvq_read(h, 0, 0, 0, 0, None, None, None) == 0  # nothing asked of an empty block
        for args in ((1, 0, 0, 0), (0, -1, 1, 0), (0, 0, -1, 0), (0, 0, 1, 0), (0, 0, 0, 2)):
            assert lib.kvq_read(h, *args, rows(p), rows(p), None) == INVALID, args
        assert lib.kvq_read(h, 0, 0, 0, 0, rows(p + 8), None, None) == INVALID
        assert lib.kvq_read(h, 0, 0, 0, 0, rows(None), None, None) == 0  # an empty tensor has no data
        assert lib.kvq_read(h, 0, 0, 0, 0, None, rows(p, t=130), None) == INVALID
        assert lib.kvq_read(None, 0, 0, 0, 0, None, None, None) == INVALID
    finally:
        kvq.kvq_free(h)


def test_python_refusals_before_any_launch(kvq):
    x = torch.zeros(1, 2, 4, 128, dtype=torch.bfloat16)
    rope = kvq.Rope(128)
    pos = torch.zeros(1, 2, dtype=torch.int64)
    with pytest.raises(ValueError):
        kvq.kvq_rope(rope, pos, None)
    with pytest.raises(ValueError):
        kvq.kvq_rope(rope, pos, x)          # not on a GPU
    with pytest.raises(TypeError):
        kvq.kvq_rope(rope, pos, x.half())   # a type the cache does not take


def test_rope_schedule_is_its_own(kvq):
    """A schedule keeps what it was made with, and copies and pickles as any other object."""
    import copy
    import pickle

    w = np.linspace(1.0, 0.1, 32)
    rope = kvq.Rope(64, layout="interleaved", inv_freq=w, magnitude=1.25)
    w[:] = 7.0
    assert rope.inv_freq[0] == 1.0
    with pytest.raises(ValueError):
        rope.inv_freq[0] = 2.0
    for other in (copy.copy(rope), copy.deepcopy(rope), pickle.loads(pickle.dumps(rope))):
        assert (other.rot_dim, other.layout, other.magnitude) == (64, "interleaved", 1.25)
        assert np.array_equal(other.inv_freq, rope.inv_freq)
        assert other._ptr.value == other.inv_freq.ctypes.data and other._code == rope._code
