"""Tree attention on Key groups whose zero is thousands of times their range, and on queries that are no numbers."""
import math

import numpy as np
import pytest
import torch

from test_gpu_operators import BF, half, kvq, make_cache, tree_inputs  # noqa: F401
from tree_accuracy import check_rms

pytestmark = pytest.mark.gpu


def exact_values(cache, mode, B, H, T):
    """What the cache holds, [B][H][T][128] in fp64 (Z + code R / (2^b - 1) with no rounding), with centres and ranges."""
    bits = cache.query(0)["bits"]
    ks, vs = torch.zeros(B, H, T, 128, dtype=torch.float64), torch.zeros(B, H, T, 128, dtype=torch.float64)
    kcen, vcen, vrange = (torch.zeros(B, H, T, 1, dtype=torch.float64) for _ in range(3))

    def put(b, j, at, exported, width):
        kc, vc, km, vm = (torch.from_numpy(np.asarray(x)) for x in exported)
        for out, cen, codes, meta in ((ks, kcen, kc, km), (vs, vcen, vc, vm)):
            r, z = (torch.from_numpy(half(meta[:, i].numpy().copy())).double()[:, None] for i in (0, 1))
            out[b, j, at] = z + codes.double() * r / (2.0 ** width - 1)
            cen[b, j, at] = z + r * 2.0 ** (width - 1) / (2.0 ** width - 1)
            if out is vs:
                vrange[b, j, at] = r

    for b in range(B):
        for j in range(H):
            own = cache.export(0, b, j)
            off = 1 if mode == "window" else 0
            put(b, j, list(range(off, off + len(own[0]))), own, bits)
            if mode == "window":
                late = cache.export_window(0, b, j)
                m = len(late[0])
                put(b, j, [0] + list(range(T - m + 1, T)), late, 16)
    ks.centre, vs.centre, vs.range = kcen, vcen, vrange
    return ks, vs


@pytest.mark.parametrize("mode", ["plain", "window"])
@pytest.mark.parametrize("fbit", [2, 4, 8, 16])
@pytest.mark.parametrize("n,G", [(6, 1), (3, 4), (4, 7), (9, 7), (16, 7)])
@pytest.mark.parametrize("Z,R", [(1000.0, 0.1), (-30000.0, 2.0), (8.0, 1e-3), (60000.0, 0.0), (1.0, 1e-4)])
def test_small_ranges_beside_large_zeros(kvq, mode, fbit, n, G, Z, R):
    """Keys of Z to Z + R in every channel: what tells tokens apart is R, and queries whose channels cancel see only that.

    Such a query's score is s sum_i q_i k_i with sum(q) = 0, so Z drops out and a Key's code, however small its range, has to
    count as R / (2^b - 1): the queries are scaled to make scores of about 3."""
    B, H, T = 1, 2, 700
    cache = kvq.KVQCache(1, B, H, 1024 * B * H * 2 * (16 * fbit + 4), [fbit], sink_window=mode == "window")
    g = torch.Generator().manual_seed(3)
    k = Z + R * torch.rand(B, T, H, 128, generator=g)
    v = torch.randn(B, T, H, 128, generator=g)
    cache.append(0, k.cuda(), v.cuda())
    ks, vs = exact_values(cache, mode, B, H, T)
    dq, dk, dv = tree_inputs(5, B, n, H, G)
    # +1 and -1 times a power of two: rounded nowhere, and they cancel to exactly zero
    sign = torch.ones(128, device="cuda")
    sign[::2] = -1.0
    q = sign[torch.argsort(dq, -1)]
    if R:
        q = q * 2.0 ** round(math.log2(3.0 / (R * 0.29)))
        dk = dk * 2.0 ** round(math.log2(R))
    got = cache.tree_attn(0, q.to(BF), dk, dv)
    check_rms(q.to(BF), dk, dv, None, ks, vs, got, mode, fbit, cancel=True)


@pytest.mark.parametrize("T", [0, 300])
@pytest.mark.parametrize("n,G", [(4, 2), (2, 3), (4, 7), (20, 3), (40, 4)])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_query_that_is_no_number_gives_none(kvq, T, n, G, bad):
    """NaN or an infinity in one channel of a query: its row is NaN in every channel, whatever the path, and no other row notices;
    a row that sees nothing is zeros as ever."""
    cache, _, ks, vs = make_cache(kvq, "plain", 2, 2, T, 4, 512)
    q, dk, dv = tree_inputs(9, 2, n, 2, G)
    mask = torch.ones(n, n, dtype=torch.bool).tril()
    mask[1] = False
    want = cache.tree_attn(0, q, dk, dv, mask.cuda())
    hit = torch.zeros(2, n, 2 * G, dtype=torch.bool, device="cuda")
    hit[0, 0, 1] = hit[1, n - 1, G] = hit[1, n // 2, 0] = hit[0, 1, 0] = True
    at = torch.arange(int(hit.sum()), device="cuda") * 37 % 128
    worse = q.clone()
    rows = worse[hit]
    rows[torch.arange(len(at), device="cuda"), at] = bad
    worse[hit] = rows
    got = cache.tree_attn(0, worse, dk, dv, mask.cuda())
    assert torch.equal(got[~hit], want[~hit])
    nothing = torch.zeros_like(hit)
    nothing[:, 1] = T == 0
    assert got[hit & ~nothing].isnan().all()
    assert (got[hit & nothing] == 0).all()
    cache.device_status()
