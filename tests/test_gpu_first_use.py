"""A cache over memory that holds anything: the error word and the ticket
counters, when the first use is captured, eager, or one and then the other."""
import gc

import pytest
import torch

import kvq_synth as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_kv_kvq_b200 import build

    build.build()
    import mixed_precision_kv_kvq_b200 as m

    m.load()
    return m


def used_memory(kvq, byte, layers=1, B=1, H=2, fbit=4):
    """A cache whose pool held other data before (every byte the same)."""
    cache = kvq.KVQCache(layers, B, H, 512 * layers * B * H * 2 * (16 * fbit + 4), [fbit] * layers)
    cache.pool.fill_(byte)
    return cache


@pytest.fixture(autouse=True)
def collected():
    """Graphs left over in reference cycles are destroyed outside captures (a destruction inside one ends it), this module's
    too before others capture."""
    gc.collect()
    yield
    gc.collect()


def status(call):
    """A call's status; no exception, and so no frame with a graph in it, is kept."""
    from mixed_precision_kv_kvq_b200 import KVQError

    try:
        call()
    except KVQError as e:
        return e.status
    return 0


def tokens(n, H=2, B=1):
    k, v = S.keys_values(3, 0, B, n, H, 0, 2)
    return k.cuda(), v.cuda()


@pytest.mark.parametrize("byte", [0x00, 0x01, 0x7F, 0xFF])
def test_what_the_pool_held_is_no_error(kvq, byte):
    cache = used_memory(kvq, byte)
    cache.device_status()
    cache.append(0, *tokens(40))
    cache.decode_attn(0, S.queries(1, 0, 0, 1, 8, 40, dtype=torch.bfloat16).cuda())
    cache.device_status()


def test_an_error_word_of_an_earlier_cache_is_not_this_ones(kvq):
    cache = used_memory(kvq, 0)
    kvq.kvq_selftest_timeout(cache.handle)
    torch.cuda.synchronize()
    per = 2 * 2 * (16 * 4 + 4)
    other = kvq.kvq_alloc(1, 1, 2, 128, 512 * per, [4], cache.pool)
    try:
        kvq.kvq_device_status(other)
    finally:
        kvq.kvq_free(other)
    assert status(cache.device_status) == 7


def test_replays_of_a_first_use_keep_an_error(kvq):
    """Two blocks appended to and attended over in one graph, captured before anything else touched the cache: a wait that
    gave up before a replay is still reported after it."""
    cache = used_memory(kvq, 0x7F, layers=2)
    k, v = tokens(9)
    q = torch.randn(1, 9, 8, 128, device="cuda").bfloat16()
    tree = torch.zeros_like(q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for layer in (0, 1):
            cache.append(layer, k, v)
            cache.tree_attn(layer, q, k, v, out=tree)
    kvq.kvq_selftest_timeout(cache.handle)
    graph.replay()
    torch.cuda.synchronize()
    assert status(cache.device_status) == 7
    graph.replay()
    cache.device_status()
    assert torch.isfinite(tree).all() and (tree != 0).any()


@pytest.mark.parametrize("how", ["decode_attn", "noalloc", "append_decode"])
def test_eager_decode_between_a_capture_and_its_replay(kvq, how):
    """The first decode is captured and does not run yet; an eager one before the replay, the replay, another graph."""
    B, H, n = 2, 2, 400
    k, v = tokens(n, H, B)
    k1, v1 = tokens(1, H, B)
    q = S.queries(1, 0, 0, B, 8, n, dtype=torch.bfloat16).cuda()

    def make(byte):
        cache = used_memory(kvq, byte, B=B, H=H)
        cache.append(0, k, v)
        return cache

    def call(cache, out, eager):
        if how == "noalloc":
            kvq.kvq_decode_attn_noalloc(cache.handle, 0, q, 128 ** -0.5, out)
        elif how == "append_decode" and not eager:
            cache.append_decode(0, k1, v1, q, out=out)
        else:
            cache.decode_attn(0, q, out=out)

    ref = make(0)
    if how == "append_decode":
        ref.append(0, k1, v1)
    want = ref.decode_attn(0, q)

    cache = make(0x7F)
    cache.workspace(0, 8)
    first, second, eager = (torch.full_like(want, 7.0) for _ in range(3))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(cache, first, False)
    if how == "append_decode":  # the captured token is not in the cache before the replay: put it there
        slot = make(0)
        slot.append(0, k1, v1)
        lo = 4096
        cache.pool[lo:].copy_(slot.pool[lo:])
    call(cache, eager, True)
    torch.cuda.synchronize()
    assert ((eager - want).abs() <= 1e-5 * want.abs().amax()).all()
    graph.replay()
    torch.cuda.synchronize()
    assert ((first - want).abs() <= 1e-5 * want.abs().amax()).all()
    again = torch.cuda.CUDAGraph()
    with torch.cuda.graph(again):
        cache.decode_attn(0, q, out=second)
    for g in (again, graph, again):
        g.replay()
    torch.cuda.synchronize()
    assert ((second - want).abs() <= 1e-5 * want.abs().amax()).all()
    cache.device_status()
