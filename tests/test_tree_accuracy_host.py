"""The accuracy check of tree attention can fail: on the CPU, outputs with the
kernels' roundings pass it, and outputs with planted mistakes do not."""
import math

import pytest
import torch

from tree_accuracy import check_rms, over

MODES = ["plain", "window", "channel"]


def cache(mode, bits, T, B=1, H=1, seed=0, loud=True):
    """Values of a block of this kind, [B][H][T][128], with their groups' centres and ranges."""
    g = torch.Generator().manual_seed(seed)
    k, v = torch.randn(B, H, T, 128, generator=g), torch.randn(B, H, T, 128, generator=g)
    if loud:
        k[..., torch.randperm(128, generator=g)[:4]] *= 20.0

    def quantized(x, dim, b):
        z = x.amin(dim, keepdim=True).half().float()
        r = (x.amax(dim, keepdim=True) - z).half().float().clamp_min(1e-6)
        top = 2.0 ** b - 1
        c = ((x - z) / r * top).round().clamp(0, top)
        return z + c * r / top, (z + r * 2.0 ** (b - 1) / top).expand_as(x), r.expand(*x.shape[:-1], r.shape[-1])

    def tokens(x):
        parts = [quantized(x, -1, bits), quantized(x, -1, 16)]
        at = torch.arange(T)
        wide = {"plain": at < 0, "window": (at == 0) | (at >= T - 128), "channel": at >= T - T % 128}[mode][:, None]
        y, c = (torch.where(wide, parts[1][i], parts[0][i]) for i in (0, 1))
        y.centre, y.range = c[..., :1], torch.where(wide, parts[1][2], parts[0][2])
        return y

    vs, ks = tokens(v), tokens(k)
    kc = ks.centre
    if mode == "channel":
        whole = T - T % 128
        blocks = k[:, :, :whole].reshape(B, H, -1, 128, 128)
        y, c, _ = quantized(blocks, 3, bits)
        old = ks
        ks = torch.cat([y.reshape(B, H, whole, 128), old[:, :, whole:]], 2)
        ks.centre = torch.cat([c.reshape(B, H, whole, 128), kc[:, :, whole:].expand(B, H, T - whole, 128)], 2)
    else:
        ks.centre = kc.expand(B, H, T, 128)
    return ks, vs


def inputs(seed, n, G, scale):
    g = torch.Generator().manual_seed(seed)
    q = (scale * torch.randn(1, n, G, 128, generator=g)).bfloat16()
    return q, torch.randn(1, n, 1, 128, generator=g).bfloat16(), torch.randn(1, n, 1, 128, generator=g).bfloat16()


def rounded(q, dk, dv, ks, vs, seen, spoil=None):
    """Attention with the roundings of the path these rows take; spoil: a change of the exact inputs first."""
    n, G = q.shape[1:3]
    narrow = n * G <= 8
    k = torch.cat([ks[0, 0], dk[0, :, 0].float()]).double()
    v = torch.cat([vs[0, 0], dv[0, :, 0].float()]).double()
    T = ks.shape[2]
    vis = torch.cat([torch.ones(n, T, dtype=torch.bool), seen], 1)
    h = lambda x: x.float().half().double()  # noqa: E731
    out = torch.zeros(1, n, G, 128, dtype=torch.float64)
    for i in range(G):
        x = q[0, :, i].double()
        if not narrow:
            x, kk, vv = h(x), h(k), h(v)
        else:
            top = x.abs().amax(1, keepdim=True)
            x, kk, vv = (x / top * 32767).round() * top / 32767, k, v
        s = torch.where(vis, x @ kk.T * 128 ** -0.5, -math.inf)
        p = torch.exp(s - s.amax(1, keepdim=True))
        if spoil is not None:
            p, vv = spoil(p, vv)
        out[0, :, i] = h(p) @ vv / p.sum(1, keepdim=True)
    return out.bfloat16()


SETTINGS = [("flat", 0.05), ("loud", 1.0)]


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("bits", [2, 4, 8, 16])
@pytest.mark.parametrize("n,G", [(5, 3), (2, 3)])
@pytest.mark.parametrize("what,scale", SETTINGS)
def test_roundings_pass(mode, bits, n, G, what, scale):
    ks, vs = cache(mode, bits, 700)
    q, dk, dv = inputs(1, n, G, scale)
    got = rounded(q, dk, dv, ks, vs, torch.ones(n, n, dtype=torch.bool).tril())
    check_rms(q, dk, dv, None, ks, vs, got, mode, bits)


@pytest.mark.parametrize("mode", MODES)
@pytest.mark.parametrize("bits", [2, 4, 8, 16])
def test_lost_and_doubled_tokens_fail(mode, bits):
    """Near-equal weights over 4,500 tokens: a group of 16, a tile, the drafted tokens; zeros; one per cent too much or too little."""
    T, n, G = 4500, 5, 2
    ks, vs = cache(mode, bits, T)
    q, dk, dv = inputs(1, n, G, 0.05)
    seen = torch.ones(n, n, dtype=torch.bool).tril()
    every = torch.arange(T + n)
    plants = [((every >= a) & (every < a + size), times) for a, size in ((0, 16), (T // 2, 16), (T - 16, 16), (2048, 128), (T, n))
              for times in (0.0, 2.0)]
    got = rounded(q, dk, dv, ks, vs, seen)
    check_rms(q, dk, dv, None, ks, vs, got, mode, bits, plant=plants)
    for tokens, times in plants:

        def spoil(p, v):
            p = p.clone()
            p[:, tokens] *= times
            return p, v

        with pytest.raises(AssertionError):
            check_rms(q, dk, dv, None, ks, vs, rounded(q, dk, dv, ks, vs, seen, spoil), mode, bits)
    for factor in (0.0, 0.99, 1.01, 1.1):
        with pytest.raises(AssertionError):
            check_rms(q, dk, dv, None, ks, vs, (got.double() * factor).bfloat16(), mode, bits)


def test_wrong_masks_scores_and_heads_fail():
    ks, vs = cache("plain", 4, 700)
    q, dk, dv = inputs(1, 5, 2, 1.0)
    seen = torch.ones(5, 5, dtype=torch.bool).tril()
    got = rounded(q, dk, dv, ks, vs, seen)
    check_rms(q, dk, dv, None, ks, vs, got, "plain", 4)
    with pytest.raises(AssertionError):
        check_rms(q, dk, dv, None, ks, vs, rounded((q.float() * 0.98).bfloat16(), dk, dv, ks, vs, seen), "plain", 4)
    with pytest.raises(AssertionError):
        check_rms(q, dk, dv, None, ks, vs, got.flip(2), "plain", 4)
    # drafted Keys as loud as the cached ones, so that what a row sees of them matters
    dk = (dk.float() * 20.0).bfloat16()
    got = rounded(q, dk, dv, ks, vs, seen)
    check_rms(q, dk, dv, None, ks, vs, got, "plain", 4)
    with pytest.raises(AssertionError):
        check_rms(q, dk, dv, seen.T, ks, vs, got, "plain", 4)


def test_limits():
    """Whole streams within 1.25, rows within 2.5 times the sum of the squares."""
    e = torch.ones(4, 128)
    assert over(e, e) == pytest.approx(0.8) and over(1.3 * e, e) > 1.0
    one = torch.zeros(400, 128)
    one[7] = 2.6
    assert over(one, torch.ones(400, 128)) > 1.0
