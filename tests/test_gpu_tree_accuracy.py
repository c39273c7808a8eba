"""Tree attention's accuracy in the root mean square, in every cache mode and
width and on both paths, with inputs where each token that could be lost or
doubled carries weight (tree_accuracy.py derives the limits)."""
import pytest
import torch

from test_gpu_operators import BF, F32, held, kvq, make_cache, randn, tree_inputs, tree_mask  # noqa: F401
from tree_accuracy import check_rms

pytestmark = pytest.mark.gpu

MODES = ["plain", "window", "channel"]
WIDTHS = [2, 4, 8, 16]


def spans(total, *pairs):
    at = torch.arange(total, device="cuda")
    return [((at >= a) & (at < a + size), times) for a, size in pairs for times in (0.0, 2.0)]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("fbit", WIDTHS)
@pytest.mark.parametrize("n,G", [(3, 4), (4, 7), (8, 8), (15, 7)])
def test_near_equal_weights(kvq, mode, fbit, n, G):
    """Every token of 2,900 counts alike, so a lost group, tile or drafted token is many times the limit."""
    B, H, T = 2, 2, 2900
    cache, lam, ks, vs = make_cache(kvq, mode, B, H, T, fbit, 4096)
    assert cache.query(0)["bits"] == fbit
    q, dk, dv = tree_inputs(n, B, n, H, G, F32 if n % 2 else BF)
    q *= 0.05
    mask = tree_mask(n, B, n=n) if G == 7 else None
    got = cache.tree_attn(0, q, dk, dv, None if mask is None else mask.cuda())
    assert torch.equal(got, cache.tree_attn(0, q, dk, dv, None if mask is None else mask.cuda()))
    plant = spans(T + n, (0, 16), (16 * 61, 16), (T - 20, 16), (T - 4, 4), (1024, 128), (T, n))
    print("relative rms error", mode, fbit, n * G, check_rms(q, dk, dv, mask, ks, vs, got, mode, fbit, lam, plant=plant))


@pytest.mark.parametrize("mode", MODES)
def test_near_equal_weights_of_wide_trees(kvq, mode):
    """More nodes than a tile of drafted tokens holds, over three blocks of rows."""
    B, H, T, n, G = 1, 2, 700, 150, 2
    cache, lam, ks, vs = make_cache(kvq, mode, B, H, T, 2, 1024)
    q, dk, dv = tree_inputs(n, B, n, H, G)
    q *= 0.05
    mask = torch.rand(B, n, n, generator=torch.Generator().manual_seed(1)) < 0.7
    got = cache.tree_attn(0, q, dk, dv, mask.cuda())
    plant = spans(T + n, (0, 16), (336, 16), (512, 128), (T, 16), (T + 112, 16), (T + 128, 16), (T + n - 6, 6))
    check_rms(q, dk, dv, mask, ks, vs, got, mode, 2, lam, plant=plant)


@pytest.mark.parametrize("fbit", WIDTHS)
@pytest.mark.parametrize("n,G", [(3, 3), (4, 7), (9, 6), (15, 7)])
def test_every_share_of_many_tiles(kvq, fbit, n, G):
    """Several streams a CTA, shares of many tiles: the ring and the buffers wrap many times in every stream.

    One token of N = 4,500 + n moves the output by 1 / N of a Value, 1.5% of the output's 1 / sqrt(N), as much as three times the
    limit (3 x 1.25 x 2^-8 for the output's rounding alone): so a group, or all drafted tokens, has to be noticed, not one."""
    B, H, T = 16, 4, 4500
    cache, lam, ks, vs = make_cache(kvq, "plain", B, H, T, fbit, 4608, lam=False)
    q, dk, dv = tree_inputs(fbit + n, B, n, H, G)
    q *= 0.05
    got = cache.tree_attn(0, q, dk, dv)
    plant = spans(T + n, (0, 16), (2048, 16), (T - 20, 16), (1024, 128), (T, n))
    streams = [(0, 0), (0, 1), (3, 2), (7, 3), (11, 1), (15, 3)]
    check_rms(q, dk, dv, None, ks, vs, got, "plain", fbit, plant=plant, streams=streams)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("fbit", WIDTHS)
@pytest.mark.parametrize("n,G", [(1, 7), (2, 4), (4, 7), (16, 7)])
@pytest.mark.parametrize("lam", [True, False])
def test_loud_channels(kvq, mode, fbit, n, G, lam):
    """Keys with loud channels and plain queries, as the cache meets them: few tokens hold most of the weight."""
    B, H, T = 2, 2, 1900
    cache, scale, ks, vs = make_cache(kvq, mode, B, H, T, fbit, 2048, lam=lam)
    q, dk, dv = tree_inputs(7 * n, B, n, H, G, F32 if n == 2 else BF)
    got = cache.tree_attn(0, q, dk, dv)
    print("relative rms error", mode, fbit, n * G, lam, check_rms(q, dk, dv, None, ks, vs, got, mode, fbit, scale))


def hadamard():
    h = torch.ones(1, 1)
    while h.shape[0] < 128:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)])
    return h


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("fbit", WIDTHS)
@pytest.mark.parametrize("n,G", [(1, 7), (2, 4), (4, 2), (8, 1), (5, 1), (3, 4), (4, 7), (9, 7), (16, 7)])
def test_chosen_tokens(kvq, mode, fbit, n, G):
    """Each row's weight lies on three cached tokens at the borders of groups, tiles, blocks and the window, and on the
    drafted tokens that it sees; it looks as hard at those that its mask hides.  Views of one projection, a mask a sequence."""
    B, H, T = 2, 2, 700
    per = B * H * 2 * (16 * fbit + 4)
    cache = kvq.KVQCache(1, B, H, 1024 * per, [fbit], sink_window=mode == "window", key_channel=mode == "channel")
    at = [0, 15, 16, 127, 128, 129, T // 3, T // 2, T - 130, T - 129, T - 128, T - 60, T - 17, T - 2, T - 1]
    g = torch.Generator().manual_seed(n)
    k, v = 0.3 * torch.randn(B, T, H, 128, generator=g), torch.randn(B, T, H, 128, generator=g)
    pattern = hadamard()[1:]
    pattern = torch.stack([torch.stack([pattern[torch.randperm(127, generator=g)] for _ in range(H)]) for _ in range(B)])  # [B][H][127][128]
    k[:, at] = 4.0 * pattern[:, :, :len(at)].transpose(1, 2)
    v[:, at] *= 2.0
    cache.append(0, k.cuda(), v.cuda())
    assert cache.query(0)["bits"] == fbit
    ks, vs = held(kvq, cache, mode, B, H, T, None)
    qkv = torch.zeros(B, n, H * G + 2 * H, 128)
    for i in range(n):
        for h in range(H * G):
            r = i * G + h % G
            mine = [(3 * r + e) % len(at) for e in range(3)]
            qkv[:, i, h] = 0.25 * (pattern[:, h // G, mine].sum(1) + pattern[:, h // G, len(at):len(at) + n].sum(1))
    qkv[:, :, H * G:H * G + H] = 4.0 * pattern[:, :, len(at):len(at) + n].transpose(1, 2)
    qkv[:, :, H * G + H:] = 2.0 * torch.randn(B, n, H, 128, generator=g)
    qkv = qkv.cuda().to(BF)
    q, dk, dv = qkv[:, :, :H * G], qkv[:, :, H * G:H * G + H], qkv[:, :, H * G + H:]
    if n % 2:
        dk, dv = dk.float(), dv.float()
    mask = tree_mask(n, B, n=n)
    got = cache.tree_attn(0, q, dk, dv, mask.cuda())
    used = at[:min(len(at), 3 * n * G)]
    plant = spans(T + n, *((t, 1) for t in used), (T, 1)) + spans(T + n, *((T + j, 1) for j in range(1, min(n, 4))))
    rel = check_rms(q, dk, dv, mask, ks, vs, got, mode, fbit, plant=plant)
    print("relative rms error", mode, fbit, n * G, rel)
    shared = mask[0].cuda()
    one = cache.tree_attn(0, q, dk, dv, shared)
    check_rms(q, dk, dv, mask[0], ks, vs, one, mode, fbit)
    if n > 2:  # the check tells masks of other sequences and the other way round apart
        for other in (mask.flip(0), mask.transpose(1, 2)):
            if not torch.equal(other, mask):
                with pytest.raises(AssertionError):
                    check_rms(q, dk, dv, other, ks, vs, got, mode, fbit)
