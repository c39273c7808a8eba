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
