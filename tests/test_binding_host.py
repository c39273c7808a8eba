"""The Python functions go by the cache's own batch and KV heads: tensors of
others are refused before anything is launched (CPU tensors and a cache over a
host buffer: nothing here reaches a GPU)."""
import pytest
import torch

from test_abi_host import _host_cache

BF = torch.bfloat16


@pytest.fixture(scope="module")
def kvq():
    from mixed_precision_kv_kvq_b200 import build

    build.build()
    import mixed_precision_kv_kvq_b200 as m

    m.load()
    return m


@pytest.fixture
def cache(kvq):
    h, pool = _host_cache(kvq, batch=2, kv_heads=3)
    yield h
    kvq.kvq_free(h)


def x(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype)


def test_dims(kvq, cache):
    assert kvq.kvq_dims(cache) == (1, 2, 3)
    assert kvq.load().kvq_dims(cache, None, None, None) == 0
    with pytest.raises(kvq.KVQError):
        kvq.kvq_dims(None)


WRONG = [(1, 4, 3, 128), (3, 4, 3, 128), (2, 4, 2, 128), (2, 4, 4, 128), (2, 4, 128)]


@pytest.mark.parametrize("shape", WRONG)
def test_read_refuses_outputs_of_another_cache(kvq, cache, shape):
    for args in ((x(*shape), None), (None, x(*shape)), (x(2, 4, 3, 128), x(*shape))):
        with pytest.raises(ValueError, match=r"must be \[2\]\[n\]\[3\]\[128\]"):
            kvq.kvq_read(cache, 0, 0, 4, *args)


@pytest.mark.parametrize("shape", WRONG)
def test_tree_refuses_inputs_of_another_cache(kvq, cache, shape):
    good = x(2, 4, 3, 128)
    for k, v in ((x(*shape), x(*shape)), (good, x(*shape)), (x(*shape), good)):
        with pytest.raises(ValueError, match=r"must be \[2\]\[n\]\[3\]\[128\]"):
            kvq.kvq_tree_attn(cache, 0, x(2, 4, 6, 128), k, v, None, 0.1, x(2, 4, 6, 128), x(1 << 16, dtype=torch.uint8))


@pytest.mark.parametrize("shape", WRONG)
def test_append_refuses_tokens_of_another_cache(kvq, cache, shape):
    with pytest.raises(ValueError, match=r"must be \[2\]\[n\]\[3\]\[128\]"):
        kvq.kvq_append(cache, 0, x(*shape), x(*shape))
    one = (shape[0], 1) + shape[2:]
    with pytest.raises(ValueError, match=r"must be \[2\]\[n\]\[3\]\[128\]"):
        kvq.kvq_append_decode(cache, 0, x(*one), x(*one), x(2, 6, 128), 0.1, x(2, 6, 128, dtype=torch.float32), x(1 << 16))


@pytest.mark.parametrize("batch", [1, 3])
def test_decode_refuses_queries_of_another_cache(kvq, cache, batch):
    q, out, ws = x(batch, 6, 128), x(batch, 6, 128, dtype=torch.float32), x(1 << 16, dtype=torch.float32)
    kv = x(2, 1, 3, 128)
    for call in (lambda: kvq.kvq_decode_attn(cache, 0, q, 0.1, out, ws), lambda: kvq.kvq_decode_attn_noalloc(cache, 0, q, 0.1, out),
                 lambda: kvq.kvq_append_decode(cache, 0, kv, kv, q, 0.1, out, ws)):
        with pytest.raises(ValueError, match=r"q must be \[2\]\[q_heads\]\[128\]"):
            call()


def test_decode_refuses_a_strided_workspace(kvq, cache):
    q, out, ws = x(2, 6, 128), x(2, 6, 128, dtype=torch.float32), x(1 << 20, dtype=torch.float32)[::2]
    kv = x(2, 1, 3, 128)
    for call in (lambda: kvq.kvq_decode_attn(cache, 0, q, 0.1, out, ws),
                 lambda: kvq.kvq_append_decode(cache, 0, kv, kv, q, 0.1, out, ws)):
        with pytest.raises(ValueError, match="workspace must be contiguous"):
            call()


class OnDevice1:
    """What the binding reads of a tensor, of one on the second GPU."""

    is_cuda, device = True, torch.device("cuda", 1)

    def __init__(self, *shape, dtype=BF):
        self.like = torch.zeros(*shape, dtype=dtype)

    def __getattr__(self, name):
        return getattr(self.like, name)


@pytest.mark.parametrize("stream", [None, 77])
def test_functions_launch_on_the_tensors_device(kvq, cache, monkeypatch, stream):
    """Device 0 is current, the tensors lie on device 1: its current stream (or the given one), with it made current."""
    calls = []

    class Guard:
        def __init__(self, device):
            calls.append(("device", device.index))

        def __enter__(self):
            calls.append("in")

        def __exit__(self, *exc):
            calls.append("out")

    class Lib:
        def kvq_read(self, *args):
            calls.append(("read", args[-1]))
            return 0

        def kvq_tree_attn(self, *args):
            calls.append(("tree", args[-1]))
            return 0

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda i: 1000 + i, raising=False)
    monkeypatch.setattr(torch.cuda, "device", Guard)
    kvq.kvq_dims(cache)
    monkeypatch.setattr(kvq, "load", lambda: Lib())
    monkeypatch.setattr(kvq, "kvq_dims", lambda c: (1, 2, 3))
    want = 1001 if stream is None else stream
    kvq.kvq_read(cache, 0, 0, 4, OnDevice1(2, 4, 3, 128), None, stream)
    assert calls == [("device", 1), "in", ("read", want), "out"]
    calls.clear()
    k = OnDevice1(2, 4, 3, 128)
    kvq.kvq_tree_attn(cache, 0, OnDevice1(2, 4, 6, 128), k, k, None, 0.1, OnDevice1(2, 4, 6, 128),
                      OnDevice1(1 << 16, dtype=torch.uint8), stream)
    assert calls == [("device", 1), "in", ("tree", want), "out"]


@pytest.mark.parametrize("which", [0, 1, 2])
def test_append_decode_refuses_host_tensors(kvq, cache, monkeypatch, which):
    monkeypatch.setattr(kvq, "load", lambda: None)  # nothing is called
    monkeypatch.setattr(kvq, "kvq_dims", lambda c: (1, 2, 3))
    kv = OnDevice1(2, 1, 3, 128)
    args = [OnDevice1(2, 6, 128), OnDevice1(2, 6, 128, dtype=torch.float32), OnDevice1(1 << 16, dtype=torch.uint8)]
    args[which] = args[which].like
    with pytest.raises(ValueError, match="must be CUDA tensors"):
        kvq.kvq_append_decode(cache, 0, kv, kv, args[0], 0.1, args[1], args[2])


def test_numbers_beyond_32_bits_are_refused(kvq, cache, monkeypatch):
    """ctypes keeps the low 32 bits of what it passes as a C int: token 2^32 would be token 0."""
    for args in ((2 ** 32 + 64,), (64, 1e4, 2 ** 32 + 1, 2.0), (64, 1e4, kvq.KVQ_ROPE_YARN, 2.0, 2 ** 32 + 4096)):
        with pytest.raises(kvq.KVQError):
            kvq.kvq_rope_freqs(*args)

    class Lib:
        def kvq_read(self, *args):
            raise AssertionError("called")

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    monkeypatch.setattr(kvq, "load", lambda: Lib())
    monkeypatch.setattr(kvq, "kvq_dims", lambda c: (1, 2, 3))
    for start in (2 ** 32, -2 ** 32, 2 ** 31):
        with pytest.raises(kvq.KVQError):
            kvq.kvq_read(cache, 0, start, 4, OnDevice1(2, 4, 3, 128), None, 77)


def test_numbers_of_other_types(kvq, cache, monkeypatch):
    """numpy's and torch's scalars are numbers, as for append and decode."""
    import numpy as np

    inv, mag = kvq.kvq_rope_freqs(np.int64(64), np.float32(10000.0), kvq.KVQ_ROPE_YARN, torch.tensor(4.0), np.int32(4096))
    want = kvq.kvq_rope_freqs(64, 10000.0, kvq.KVQ_ROPE_YARN, 4.0, 4096)
    assert np.array_equal(inv, want[0]) and mag == want[1]
    calls = []

    class Lib:
        def kvq_read(self, *args):
            calls.append(args[2:4])
            return 0

        def kvq_tree_attn(self, *args):
            calls.append(args[10])
            return 0

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 1, raising=False)
    monkeypatch.setattr(kvq, "load", lambda: Lib())
    monkeypatch.setattr(kvq, "kvq_dims", lambda c: (1, 2, 3))
    k = OnDevice1(2, 4, 3, 128)
    kvq.kvq_read(cache, 0, np.int64(7), torch.tensor(4), k, None, 77)
    for scale in (np.float32(0.5), torch.tensor(0.5), 0.5):
        kvq.kvq_tree_attn(cache, 0, OnDevice1(2, 4, 6, 128), k, k, None, scale, OnDevice1(2, 4, 6, 128),
                          OnDevice1(1 << 16, dtype=torch.uint8), 77)
    assert calls == [(7, 4), 0.5, 0.5, 0.5] and all(type(x) in (tuple, float) for x in calls)
    assert all(type(x) is int for x in calls[0])
