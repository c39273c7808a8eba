"""Calls of the operators' functions that are refused, or valid and unusual, on the GPU."""
import pytest
import torch

import kvq_synth as S

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module")
def kvq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_kv_kvq_b200 import build

    build.build()
    import mixed_precision_kv_kvq_b200 as m

    m.load()
    return m


def filled(kvq, B, H, T=300, fbit=4, **options):
    cache = kvq.KVQCache(1, B, H, 512 * B * H * 2 * (16 * fbit + 4), [fbit], **options)
    k, v = S.keys_values(5, 0, B, T, H, 0, 2)
    cache.append(0, k.cuda(), v.cuda())
    return cache


def rand(seed, *shape, dtype=BF):
    return torch.randn(*shape, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(dtype)


def test_functions_refuse_other_batches_and_heads(kvq):
    cache = filled(kvq, 2, 2)
    room = torch.zeros(2, 20, 4, 128, device="cuda", dtype=BF)
    for out in (room[:1, :10, :2], room[:, :10, :1], room[:, :10, :3]):
        with pytest.raises(ValueError):
            kvq.kvq_read(cache.handle, 0, 0, 10, out, None)
        with pytest.raises(ValueError):
            cache.read(0, 0, 10, v_out=out)
    torch.cuda.synchronize()
    assert (room == 0).all()
    kvq.kvq_read(cache.handle, 0, 0, 10, room[:, :10, :2], None)
    assert torch.equal(room[:, :10, :2], cache.read(0, 0, 10)[0]) and (room[:, 10:] == 0).all() and (room[:, :, 2:] == 0).all()
    q, k = rand(1, 2, 4, 6, 128), rand(2, 2, 4, 2, 128)
    ws = torch.empty(kvq.kvq_tree_workspace(cache.handle, 0, 6, 4), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(q)
    for kk in (k[:1], k[:, :, :1], rand(3, 2, 4, 3, 128)):
        with pytest.raises(ValueError):
            kvq.kvq_tree_attn(cache.handle, 0, q, kk, kk, None, 0.1, out, ws)
    with pytest.raises(ValueError):  # every second byte of a workspace
        wide = torch.empty(2 * ws.numel(), dtype=torch.uint8, device="cuda")
        kvq.kvq_tree_attn(cache.handle, 0, q, k, k, None, 0.1, out, wide[::2])
    torch.cuda.synchronize()
    assert (out == 0).all()
    kvq.kvq_tree_attn(cache.handle, 0, q, k, k, None, 0.1, out, ws)
    assert torch.equal(out, cache.tree_attn(0, q, k, k, sm_scale=0.1))


def odd(t, *dims):
    """The same elements with strides of 1 in the given dimensions, each of one element."""
    strides = list(t.stride())
    for d in dims:
        assert t.shape[d] == 1
        strides[d] = 1
    return torch.as_strided(t, t.shape, strides, t.storage_offset())


@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("B,n,H,dims", [(1, 5, 2, (0,)), (2, 1, 2, (1,)), (2, 5, 1, (2,)), (1, 1, 1, (0, 1, 2))])
def test_strides_of_single_elements_are_free(kvq, dtype, B, n, H, dims):
    """A dimension of one element may have any stride: [b][n][1][128] made of a transposed [b][n][128][1], a slice of one
    sequence or token."""
    cache = filled(kvq, B, H)
    k, v = rand(2, B, n, H, 128, dtype=dtype), rand(3, B, n, H, 128, dtype=dtype)
    room = torch.zeros(B, n, H, 128, device="cuda", dtype=dtype)
    want = cache.read(0, 3, n, dtype=dtype)
    got = cache.read(0, 3, n, k_out=odd(room, *dims), v_out=odd(torch.zeros_like(room), *dims))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and torch.equal(room, want[0])
    for G in (1, 8):
        q = rand(1, B, n, H * G, 128)
        want = cache.tree_attn(0, q, k, v)
        qd = [d for d in dims if q.shape[d] == 1]
        assert torch.equal(cache.tree_attn(0, odd(q, *qd), odd(k, *dims), odd(v, *dims)), want)
    pos = torch.arange(n, device="cuda")
    for layout in ("half", "interleaved"):
        rope = kvq.Rope(128, layout=layout)
        want = kvq.kvq_rope(rope, pos, k, v)
        out = torch.zeros_like(k)
        assert torch.equal(kvq.kvq_rope(rope, pos, odd(k, *dims), odd(v, *dims), q_out=odd(out, *dims))[0], want[0])
        assert torch.equal(out, want[0])


@pytest.mark.parametrize("T", [0, 300, 2900])
@pytest.mark.parametrize("n,G", [(1, 7), (4, 2), (4, 7), (16, 7), (40, 7)])
def test_tree_into_its_own_queries(kvq, T, n, G):
    """out may be q itself: rows cut over several CTAs, rows of one, and the path of up to 8 rows; eager and replayed."""
    B, H = 2, 2
    cache = kvq.KVQCache(1, B, H, 4096 * B * H * 2 * (16 * 4 + 4), [4])
    if T:
        k, v = S.keys_values(5, 0, B, T, H, 0, 2)
        cache.append(0, k.cuda(), v.cuda())
    q, k, v = rand(1, B, n, H * G, 128), rand(2, B, n, H, 128), rand(3, B, n, H, 128)
    want = cache.tree_attn(0, q, k, v)
    for _ in range(5):
        own = q.clone()
        assert cache.tree_attn(0, own, k, v, out=own) is own
        assert torch.equal(own, want)
    own = q.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.tree_attn(0, own, k, v, out=own)
    for _ in range(3):
        own.copy_(q)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(own, want)


@pytest.mark.parametrize("n,G", [(1, 7), (4, 7), (16, 7)])
def test_tree_of_broadcast_queries_and_drafts(kvq, n, G):
    """Every sequence drafts the same tokens: q, k and v expanded over the batch, as copies of them."""
    B, H = 3, 2
    cache = filled(kvq, B, H)
    q, k, v = (rand(i, 1, n, h, 128).expand(B, n, h, 128) for i, h in ((1, H * G), (2, H), (3, H)))
    assert torch.equal(cache.tree_attn(0, q, k, v), cache.tree_attn(0, q.contiguous(), k.contiguous(), v.contiguous()))
    rope, pos = kvq.Rope(128), torch.arange(n, device="cuda")
    a, b = kvq.kvq_rope(rope, pos, q, k), kvq.kvq_rope(rope, pos[None].expand(B, n), q.contiguous(), k.contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("mode", [{}, {"sink_window": True}, {"key_channel": True}])
def test_calls_at_once_on_several_streams(kvq, mode):
    """Reading, both tree paths and a rotation run at once on streams of their own, over a cache that none of them changes."""
    B, H = 2, 2
    cache = kvq.KVQCache(1, B, H, 4096 * B * H * 2 * (16 * 2 + 4), [2], **mode)
    k, v = S.keys_values(5, 0, B, 3000, H, 0, 2)
    cache.append(0, k.cuda(), v.cuda())
    rope, pos = kvq.Rope(128), torch.arange(12, device="cuda")
    q, dk, dv = rand(1, B, 12, 2 * 7, 128), rand(2, B, 12, H, 128), rand(3, B, 12, H, 128)
    calls = [lambda s: cache.read(0, 100, 2500, stream=s), lambda s: (cache.tree_attn(0, q, dk, dv, stream=s),),
             lambda s: (cache.tree_attn(0, q[:, :1], dk[:, :1], dv[:, :1], stream=s),), lambda s: kvq.kvq_rope(rope, pos, q, dk, stream=s)]
    want = [c(None) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[c(s) for c, s in zip(calls, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    for row in got:
        for a, b in zip(row, want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
    cache.device_status()
