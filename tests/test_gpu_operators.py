"""Rotary positions, tree attention and reading back on the GPU, against plain
64-bit forms.

Tolerances.  A rounding to type t is off by at most half a step, u_t =
finfo(t).eps / 2 relative to the value (bf16 2^-8, fp16 2^-11, fp32 2^-24).
 * rotary: y = (x0 c - x1 s) mag in fp32: the angle is off by 2 pi 2^-26 rad
   (and the 64-bit form's own product by angle 2^-53 <= 2.4e-7 at 2^31), c and
   s by 2 steps (2^-22), three fp32 roundings: below 1e-6 (|x0| + |x1|) mag in
   all, plus u_t |y|.
 * read: every step is one IEEE fp32 operation, so fp32 outputs are equal and
   bf16 outputs are those values rounded.
 * tree, u = u_fp16 and w the weights.  Cached values go through their group's
   centre c = Z + R 2^(b-1) / (2^b - 1): centre and value are each rounded
   once, the 16-bit codes once more and the 16-bit range of a block that has
   other widths once more, the latter two relative to |v - c| <= |v| + |c|; p is
   rounded once (2^-25 absolute below 2^-14, against a largest p of about 1).  So
   the output is off by u sum_t w_t (4 |v_t| + 3 |c_t|) + T 2^-25 max |v|.
   A score sum_c q'_c k_c has q' rounded, and k like a value but for the range:
   delta = u sum_c |q'_c| (3 |k_c| + 2 |c|), c the centre of the Key's group (of
   its channel's block with per-channel groups), plus 2e-4 for the fp32 sums
   and the exponential; weights then change by at most e^(2 delta) - 1 relative.
   Up to 8 rows (n G) go through the decode kernel: its 15-bit query is finer,
   but its Value codes enter the MMA uncentred as subnormals, whose products are
   off by up to 2^-12 of the sum of the terms' sizes, sum_t w_t R_t (the
   decode kernel's measured bound is 1.8e-4 < 2^-12), p R is rounded once
   (u |v - c| <= u (|v| + |c|)), and its p may exceed the largest by 2^8 less.
   The output is rounded once to bf16:
   |o - o*| <= u_bf16 |o*| 1.02 + 1.02 ((e^(2 delta) - 1) sum_t w_t |v_t| + the
   above) + 1e-6 (1.02: products of these, and second orders)."""
import math

import numpy as np
import pytest
import torch

import kvq_synth as S

pytestmark = pytest.mark.gpu

U16, UBF = 2.0 ** -11, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def kvq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from mixed_precision_kv_kvq_b200 import build

    build.build()
    import mixed_precision_kv_kvq_b200 as m

    m.load()
    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(seed, *shape, dtype=BF):
    return torch.randn(*shape, generator=gen(seed), device="cuda").to(dtype)


# ------------------------------------------------------------------ rotary

def rope_exact(rope, pos, x):
    half = rope.rot_dim // 2
    inv = torch.tensor(rope.inv_freq, device="cuda")
    ang = (pos if pos.dim() == 2 else pos.expand(x.shape[0], -1)).double()[:, :, None, None] * inv
    c, s = ang.cos() * rope.magnitude, ang.sin() * rope.magnitude
    y = x.double().clone()
    if rope.layout == "half":
        i, j = slice(0, half), slice(half, 2 * half)
    else:
        i, j = slice(0, 2 * half, 2), slice(1, 2 * half, 2)
    a, b = x[..., i].double(), x[..., j].double()
    y[..., i], y[..., j] = a * c - b * s, b * c + a * s
    size = torch.zeros_like(y)
    size[..., i] = size[..., j] = (a.abs() + b.abs()) * abs(rope.magnitude)
    return y, size


def rope_check(rope, pos, x, got):
    y, size = rope_exact(rope, pos, x)
    tol = torch.finfo(x.dtype).eps / 2 * y.abs() + 1.01e-6 * size
    assert got.dtype == x.dtype and got.shape == x.shape
    assert ((got.double() - y).abs() <= tol).all()
    assert torch.equal(got[..., rope.rot_dim:], x[..., rope.rot_dim:])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("rot", [2, 6, 24, 40, 64, 96, 128])
def test_rope_layouts_and_parts(kvq, dtype, layout, rot):
    rope = kvq.Rope(rot, layout=layout)
    q, k = randn(1, 2, 5, 6, 128, dtype=dtype), randn(2, 2, 5, 2, 128, dtype=dtype)
    pos = torch.randint(0, 4000, (2, 5), generator=gen(3), device="cuda")
    qo, ko = kvq.kvq_rope(rope, pos, q, k)
    rope_check(rope, pos, q, qo)
    rope_check(rope, pos, k, ko)


@pytest.mark.parametrize("scaling", ["none", "linear", "ntk", "yarn"])
@pytest.mark.parametrize("first", [0, 131072, 2 ** 31 - 4100])
def test_rope_far_positions(kvq, scaling, first):
    rope = kvq.Rope(128, scaling=scaling, factor=8.0 if scaling != "none" else 1.0, original_tokens=4096)
    q = randn(4, 1, 4099, 3, 128, dtype=F32)
    pos = torch.arange(first, first + 4099, device="cuda")[None]
    qo, ko = kvq.kvq_rope(rope, pos, q)
    assert ko is None
    rope_check(rope, pos, q, qo)
    p32 = pos.to(torch.int32)
    assert torch.equal(kvq.kvq_rope(rope, p32, q)[0], qo)
    assert torch.equal(kvq.kvq_rope(rope, p32[0], q)[0], qo)


def test_rope_negative_positions_turn_back(kvq):
    rope = kvq.Rope(128, layout="interleaved")
    q = randn(5, 2, 7, 4, 128, dtype=F32)
    pos = torch.randint(0, 100000, (2, 7), generator=gen(6), device="cuda")
    back = kvq.kvq_rope(rope, -pos, kvq.kvq_rope(rope, pos, q)[0])[0]
    size = q[..., 0::2].abs() + q[..., 1::2].abs()
    assert ((back - q).abs() <= 4.1e-6 * size.repeat_interleave(2, -1)).all()  # two turns, each 1e-6 of up to twice the size


@pytest.mark.parametrize("offset", [0, 1, 2, 4, 8])
def test_rope_strided_views_and_alignment(kvq, offset):
    """q and k as slices of a fused projection, [b][h][t][d] outputs, rows off 16 bytes."""
    rope = kvq.Rope(128)
    flat = randn(7, 3 * 9 * 8 * 128 + offset)
    qkv = flat[offset:].view(3, 9, 8, 128)
    q, k = qkv[:, :, :4], qkv[:, :, 4:6]
    pos = torch.randint(0, 4000, (9, 3), generator=gen(8), device="cuda").t()
    qo = torch.zeros(3, 4, 9, 128, dtype=BF, device="cuda").transpose(1, 2)
    ko = torch.zeros(3, 9, 2, 128, dtype=BF, device="cuda")
    keep = flat.clone()
    a, b = kvq.kvq_rope(rope, pos, q, k, qo, ko)
    assert a is qo and b is ko and torch.equal(flat, keep)
    rope_check(rope, pos, q, qo)
    rope_check(rope, pos, k, ko)
    # in place
    kvq.kvq_rope(rope, pos, q, k, q, k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(qkv[:, :, 6:], keep[offset:].view(3, 9, 8, 128)[:, :, 6:])


def test_rope_interleaved_refuses_half_pairs(kvq):
    x = randn(9, 1 * 2 * 1 * 128 + 1)[1:].view(1, 2, 1, 128)
    with pytest.raises(kvq.KVQError):
        kvq.kvq_rope(kvq.Rope(128, layout="interleaved"), torch.zeros(1, 2, dtype=torch.int64, device="cuda"), x)


def test_rope_streams_graphs_and_nothing(kvq):
    rope = kvq.Rope(64)
    q = randn(10, 2, 3, 4, 128)
    pos = torch.arange(3, device="cuda")
    want = kvq.kvq_rope(rope, pos, q)[0]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = kvq.kvq_rope(rope, pos, q, stream=side)[0]
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvq.kvq_rope(rope, pos, q, q_out=out)
    q.copy_(randn(11, 2, 3, 4, 128))
    graph.replay()
    torch.cuda.synchronize()
    rope_check(rope, pos[None].expand(2, 3), q, out)
    empty = torch.empty(2, 0, 4, 128, dtype=BF, device="cuda")
    assert kvq.kvq_rope(rope, torch.empty(0, dtype=torch.int64, device="cuda"), empty)[0].shape == empty.shape
    none = torch.empty(2, 3, 0, 128, dtype=BF, device="cuda")
    assert kvq.kvq_rope(rope, pos, none, q)[1].shape == q.shape


def test_rope_refusals(kvq):
    rope = kvq.Rope(128)
    q = randn(12, 2, 3, 4, 128)
    pos = torch.arange(3, device="cuda")
    for bad in (lambda: kvq.kvq_rope(rope, pos.float(), q), lambda: kvq.kvq_rope(rope, pos[:2], q),
                lambda: kvq.kvq_rope(rope, pos, q, q[:, :2]), lambda: kvq.kvq_rope(rope, pos, q[..., :64]),
                lambda: kvq.kvq_rope(rope, pos, q, q_out=q[:, :, :2]), lambda: kvq.kvq_rope(rope, pos.cpu(), q),
                lambda: kvq.kvq_rope(rope, pos, q.transpose(2, 3).contiguous().transpose(2, 3)),
                lambda: kvq.kvq_rope(rope, pos, q, k_out=q)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: kvq.kvq_rope(rope, pos, q.half()), lambda: kvq.kvq_rope(rope, pos, q, q.float())):
        with pytest.raises(TypeError):
            bad()


# ------------------------------------------------------ caches of the tests

MODES = ["plain", "window", "channel"]


def make_cache(kvq, mode, B, H, T, fbit, n_f, seed=0, lam=True, direct=False, chunk=0, sample=None):
    """A cache of T random tokens (Keys with loud channels) and the values it holds, fp32 [B][H][T][128] each, by the
    codes and meta that export gives (lambda undone).  ks.centre, vs.centre: the centres of their groups.
    sample: of the one stream (b, h) only."""
    per = B * H * 2 * (16 * fbit + 4)
    cache = kvq.KVQCache(1, B, H, n_f * per, [fbit], sink_window=mode == "window", key_channel=mode == "channel")
    k, v = S.keys_values(seed, 0, B, max(T, 1), H, 0, 4, dtype=torch.float32)
    k, v = k[:, :T], v[:, :T]
    scale = None
    if lam:
        scale = (k.abs().amax((0, 1)).sqrt().clamp_min(0.05) if T else torch.ones(H, 128)).float().contiguous()
        cache.set_lambda(0, scale)
    if direct:
        cache.set_shift_mode(0, kvq.KVQ_SHIFT_DIRECT)
    at = 0
    while at < T:
        n = min(chunk or T, T - at)
        cache.append(0, k[:, at:at + n].contiguous().cuda(), v[:, at:at + n].contiguous().cuda())
        at += n
    return (cache, scale) + held(kvq, cache, mode, B, H, T, scale, sample)


def half(bits):
    return bits.view(np.float16).astype(np.float32)


def held(kvq, cache, mode, B, H, T, scale, sample=None):
    bits = cache.query(0)["bits"]
    streams = [sample] if sample else [(b, j) for b in range(B) for j in range(H)]
    if sample:
        B = H = 1
    ks, vs = np.zeros((B, H, T, 128), np.float32), np.zeros((B, H, T, 128), np.float32)

    kcen, vcen = np.zeros((B, H, T, 128), np.float32), np.zeros((B, H, T, 1), np.float32)
    vrange = np.zeros((B, H, T, 1), np.float32)

    def centre(r, z, b):
        return z + r * (2.0 ** (b - 1) / (2.0 ** b - 1))

    def values(codes, r, z, b):
        return (codes.astype(np.float32) * (r / np.float32(2 ** b - 1)) + z).astype(np.float32)

    for sb, sj in streams:
        b, j = (0, 0) if sample else (sb, sj)
        kc, vc, km, vm = cache.export(0, sb, sj)
        n = len(kc)
        off = 1 if mode == "window" else 0
        if n:
            if mode == "channel":
                kr = np.repeat(half(km[:, 0]).reshape(-1, 128), 128, 0)
                kz = np.repeat(half(km[:, 1]).reshape(-1, 128), 128, 0)
            else:
                kr, kz = half(km[:, 0])[:, None], half(km[:, 1])[:, None]
            ks[b, j, off:off + n] = values(kc, kr, kz, bits)
            vs[b, j, off:off + n] = values(vc, half(vm[:, 0])[:, None], half(vm[:, 1])[:, None], bits)
            kcen[b, j, off:off + n] = centre(kr, kz, bits)
            vcen[b, j, off:off + n] = centre(half(vm[:, 0])[:, None], half(vm[:, 1])[:, None], bits)
            vrange[b, j, off:off + n] = half(vm[:, 0])[:, None]
        if mode != "plain":
            kc, vc, km, vm = cache.export_window(0, sb, sj)
            m = len(kc)
            at = list(range(T - m, T)) if mode == "channel" else ([0] + list(range(T - m + 1, T)) if m else [])
            ks[b, j, at] = values(kc, half(km[:, 0])[:, None], half(km[:, 1])[:, None], 16)
            vs[b, j, at] = values(vc, half(vm[:, 0])[:, None], half(vm[:, 1])[:, None], 16)
            kcen[b, j, at] = centre(half(km[:, 0])[:, None], half(km[:, 1])[:, None], 16)
            vcen[b, j, at] = centre(half(vm[:, 0])[:, None], half(vm[:, 1])[:, None], 16)
            vrange[b, j, at] = half(vm[:, 0])[:, None]
    if scale is not None:
        ks = ks * scale.numpy()[None, :, None, :]
        kcen = kcen * scale.numpy()[None, :, None, :]
    ks, vs = torch.from_numpy(ks), torch.from_numpy(vs)
    ks.centre, vs.centre, vs.range = torch.from_numpy(kcen), torch.from_numpy(vcen), torch.from_numpy(vrange)
    return ks, vs


# ------------------------------------------------------------- reading back

CASES = [("plain", 700, 2, 1024), ("plain", 333, 16, 512), ("plain", 1024, 2, 1024), ("plain", 1500, 4, 1536),
         ("plain", 1000, 8, 1024), ("plain", 1, 4, 512), ("plain", 17, 2, 512),
         ("window", 1, 2, 512), ("window", 100, 4, 512), ("window", 129, 2, 512), ("window", 130, 2, 512),
         ("window", 700, 2, 1024), ("window", 600, 8, 512),
         ("channel", 100, 2, 1024), ("channel", 128, 4, 1024), ("channel", 1100, 2, 1024), ("channel", 700, 8, 1024)]


@pytest.mark.parametrize("mode,T,fbit,n_f", CASES)
@pytest.mark.parametrize("lam", [True, False])
def test_read_equals_the_codes(kvq, mode, T, fbit, n_f, lam):
    cache, _, ks, vs = make_cache(kvq, mode, 2, 3, T, fbit, n_f, lam=lam, direct=T == 700)
    k, v = cache.read(0, dtype=F32)
    assert k.shape == (2, T, 3, 128)
    assert torch.equal(k.cpu().transpose(1, 2), ks) and torch.equal(v.cpu().transpose(1, 2), vs)
    g = torch.Generator().manual_seed(T)
    for _ in range(4):
        a = int(torch.randint(0, T, (1,), generator=g))
        n = int(torch.randint(1, T - a + 1, (1,), generator=g))
        k, v = cache.read(0, a, n)
        assert torch.equal(k.cpu().transpose(1, 2), ks[:, :, a:a + n].bfloat16())
        assert torch.equal(v.cpu().transpose(1, 2), vs[:, :, a:a + n].bfloat16())
    assert cache.read(0, T, 0)[0].shape == (2, 0, 3, 128)


def test_read_into_views(kvq):
    """One output only, [b][h][t][d] layout, rows around the range left as they were, another stream, a replayed graph."""
    cache, _, ks, vs = make_cache(kvq, "plain", 2, 2, 700, 4, 1024)
    room = torch.full((2, 2, 40, 128), 7.0, device="cuda")
    view = room[:, :, 5:30].transpose(1, 2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    k, v = cache.read(0, 300, 25, k_out=view, stream=side)
    side.synchronize()
    assert v is None and k is view
    assert torch.equal(room[:, :, 5:30].cpu(), ks[:, :, 300:325])
    assert (room[:, :, :5] == 7).all() and (room[:, :, 30:] == 7).all()
    out = torch.zeros(2, 25, 2, 128, device="cuda", dtype=BF)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cache.read(0, 300, 25, v_out=out)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out.cpu().transpose(1, 2), vs[:, :, 300:325].bfloat16())
    for bad in (lambda: cache.read(0, 0, 701), lambda: cache.read(0, -1, 2), lambda: cache.read(1, 0, 1)):
        with pytest.raises(kvq.KVQError):
            bad()
    for bad in (lambda: cache.read(0, 0, 24, v_out=out), lambda: cache.read(0, 0, -1), lambda: cache.read(0, 701),
                lambda: cache.read(0, 0, 25, v_out=out[:, :, :1])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        cache.read(0, 0, 25, v_out=out.half())


def test_read_appended_again_is_stable(kvq):
    """Reading a 16-bit block and appending it to another gives back the same values up to two 16-bit quantizations."""
    cache, scale, ks, vs = make_cache(kvq, "plain", 1, 2, 300, 16, 512)
    k, v = cache.read(0, dtype=F32)
    other = kvq.KVQCache(1, 1, 2, 512 * 2 * 2 * (16 * 16 + 4), [16])
    other.set_lambda(0, scale)
    other.append(0, k, v)
    k2, v2 = other.read(0, dtype=F32)
    span = (v.amax(-1) - v.amin(-1))[..., None]
    # half a 16-bit step, and the binary16 range rounded up by at most 2^-10 of itself
    assert ((v2 - v).abs() <= 0.6 * span * 1.01 / 65535 + 2.0 ** -22 * v.abs()).all()


# --------------------------------------------------------- tree attention

def tree_mask(seed, *lead, n):
    g = torch.Generator().manual_seed(seed)
    m = torch.zeros(*lead, n, n, dtype=torch.bool)
    for i in range(n):
        for at in np.ndindex(*lead) if lead else [()]:
            p = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
            if p >= 0:
                m[at + (i,)] = m[at + (p,)]
            m[at + (i, i)] = True
    return m


def tree_check(q, dk, dv, mask, ks, vs, got, sm_scale=128 ** -0.5):
    """q [B][n][Hq][128], dk, dv [B][n][H][128], ks, vs [B][H][T][128]; mask bool [n][n], [B][n][n] or None."""
    B, n, Hq, _ = q.shape
    H = dk.shape[2]
    G = Hq // H
    dev = "cuda"
    seen = torch.ones(n, n, dtype=torch.bool).tril() if mask is None else mask.bool().cpu()
    seen = seen.expand(B, n, n).to(dev)
    kc, vc, vr = (x.to(dev).double().abs() for x in (ks.centre, vs.centre, vs.range))
    ks, vs = ks.to(dev).double(), vs.to(dev).double()
    T = ks.shape[2]
    bad = torch.full((), -math.inf, dtype=torch.float64, device=dev)
    for b in range(B):
        for j in range(H):
            kk = torch.cat([ks[b, j], dk[b, :, j].double()])
            vv = torch.cat([vs[b, j], dv[b, :, j].double()])
            vis = torch.cat([torch.ones(n, T, dtype=torch.bool, device=dev), seen[b]], 1)
            kk, vv = torch.nan_to_num(kk, 0, 0, 0), torch.nan_to_num(vv, 0, 0, 0)
            kerr = 3 * kk.abs()
            kerr[:T] += 2 * kc[b, j]
            verr = 4 * vv.abs()
            verr[:T] += 3 * vc[b, j]
            if n * G <= 8 and T:
                verr[:T] += 2.0 ** -12 / U16 * vr[b, j]
            for g in range(G):
                qq = q[b, :, j * G + g].double()
                s = torch.where(vis, sm_scale * (qq @ kk.T), bad)
                size = torch.where(vis, abs(sm_scale) * (qq.abs() @ kerr.T), 0.0).amax(1, keepdim=True)
                w = torch.softmax(s, -1)
                empty = ~vis.any(1)
                w[empty] = 0.0
                o = w @ vv
                delta = U16 * size + 2e-4
                off = (torch.exp(2 * delta) - 1) * (w @ vv.abs()) + U16 * (w @ verr) + (T + n) * 2.0 ** -25 * vv.abs().max()
                tol = UBF * 1.02 * o.abs() + 1.02 * off + 1e-6
                y = got[b, :, j * G + g].double()
                assert torch.isfinite(y).all(), (b, j, g)
                off = (y - o).abs() - tol
                assert (off <= 0).all(), (b, j, g, float(off.max()), torch.nonzero(off > 0)[:3].tolist())
                assert (y[empty] == 0).all()


def tree_inputs(seed, B, n, H, G, dtype=BF):
    q = randn(seed, B, n, H * G, 128)
    dk, dv = randn(seed + 1, B, n, H, 128, dtype=dtype), randn(seed + 2, B, n, H, 128, dtype=dtype)
    return q, dk, dv


@pytest.mark.parametrize("mode,T,fbit,n_f", CASES + [("plain", 0, 4, 512), ("window", 0, 4, 512), ("channel", 0, 4, 1024)])
@pytest.mark.parametrize("n,G,masked", [(1, 1, False), (3, 7, True), (16, 8, True), (37, 5, False)])
def test_tree_caches(kvq, mode, T, fbit, n_f, n, G, masked):
    B, H = 2, 3
    cache, _, ks, vs = make_cache(kvq, mode, B, H, T, fbit, n_f, lam=n != 3, direct=T == 700)
    q, dk, dv = tree_inputs(T + n, B, n, H, G, BF if n % 2 else F32)
    mask = tree_mask(n, B, n=n) if masked else None
    out = cache.tree_attn(0, q, dk, dv, mask.cuda() if masked else None)
    assert out.dtype == BF and out.shape == q.shape
    tree_check(q, dk, dv, mask, ks, vs, out)
    cache.device_status()


@pytest.mark.parametrize("n,G", [(1, 2), (1, 8), (2, 8), (4, 8), (6, 8), (8, 8), (9, 7), (12, 8), (16, 8), (17, 8), (64, 1),
                                 (65, 1), (128, 1), (129, 2), (257, 1), (300, 5)])
def test_tree_rows(kvq, n, G):
    """Every number of query rows around the row blocks' borders, over several splits."""
    cache, _, ks, vs = make_cache(kvq, "plain", 1, 2, 2900, 4, 4096, lam=True)
    q, dk, dv = tree_inputs(n, 1, n, 2, G)
    mask = tree_mask(n, n=n).to(torch.uint8) * 3
    out = cache.tree_attn(0, q, dk, dv, mask.cuda())
    tree_check(q, dk, dv, mask, ks, vs, out)


@pytest.mark.parametrize("T", [1, 15, 16, 127, 128, 129, 255, 1023, 2047, 2048, 2049, 4095, 4096])
@pytest.mark.parametrize("fbit", [2, 4])
def test_tree_lengths(kvq, T, fbit):
    """Partial groups, tiles that are half full after a shrink, blocks that end inside a tile."""
    cache, _, ks, vs = make_cache(kvq, "plain", 1, 1, T, fbit, 4096, chunk=999)
    q, dk, dv = tree_inputs(T, 1, 5, 1, 6)
    out = cache.tree_attn(0, q, dk, dv)
    tree_check(q, dk, dv, None, ks, vs, out)


@pytest.mark.parametrize("fbit", [2, 4, 8, 16])
@pytest.mark.parametrize("n,G", [(1, 5), (4, 7), (9, 6), (15, 7), (40, 7)])
def test_tree_many_tiles(kvq, fbit, n, G):
    """Shares of many tiles and several streams a CTA at every width and division of the warps: the ring and the
    buffers wrap many times, and drafted tiles (an odd number of them here) change which buffer a tile takes."""
    B, H, T = 16, 4, 4500
    cache, _, ks, vs = make_cache(kvq, "plain", B, H, T, fbit, 4608, lam=False, sample=(B - 1, H - 1))
    q, dk, dv = tree_inputs(fbit + n, B, n, H, G)
    outs = [cache.tree_attn(0, q, dk, dv) for _ in range(3)]
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])
    one = slice(B - 1, B), slice(H - 1, H)
    tree_check(q[one[0], :, (H - 1) * G:], dk[one[0], :, one[1]], dv[one[0], :, one[1]], None, ks, vs,
               outs[0][one[0], :, (H - 1) * G:])
    cache.device_status()


def test_tree_long(kvq):
    """A long context and more streams than one wave; the largest tree."""
    cache, _, ks, vs = make_cache(kvq, "plain", 3, 5, 20000, 2, 20480)
    for n in (1, 13):
        q, dk, dv = tree_inputs(n, 3, n, 5, 7)
        tree_check(q, dk, dv, None, ks, vs, cache.tree_attn(0, q, dk, dv))
    cache, _, ks, vs = make_cache(kvq, "plain", 1, 1, 600, 8, 1024)
    q, dk, dv = tree_inputs(5, 1, 1024, 1, 3)
    mask = torch.rand(1024, 1024, generator=torch.Generator().manual_seed(1)) < 0.3
    tree_check(q, dk, dv, mask, ks, vs, cache.tree_attn(0, q, dk, dv, mask.cuda()))


def test_tree_growing_scores(kvq):
    """Scores that rise and fall by hundreds along the context: the running maximum moves many times."""
    B, H, T = 1, 2, 1500
    cache = kvq.KVQCache(1, B, H, 2048 * B * H * 2 * (16 * 8 + 4), [8])
    k = torch.zeros(B, T, H, 128)
    k[..., 0] = torch.linspace(-30, 40, T)[None, :, None]
    k[..., 1] = torch.linspace(50, -50, T)[None, :, None]
    k += 0.1 * torch.randn(B, T, H, 128, generator=torch.Generator().manual_seed(0))
    v = torch.randn(B, T, H, 128, generator=torch.Generator().manual_seed(1))
    cache.append(0, k.cuda(), v.cuda())
    ks, vs = held(kvq, cache, "plain", B, H, T, None)
    q, dk, dv = tree_inputs(3, B, 6, H, 4)
    q *= 0.3
    q[:, 0::3, :, 0] = 60.0
    q[:, 1::3, :, 1] = -60.0
    tree_check(q, dk, dv, None, ks, vs, cache.tree_attn(0, q, dk, dv))


@pytest.mark.parametrize("T", [0, 300])
def test_tree_rows_that_see_nothing(kvq, T):
    cache, _, ks, vs = make_cache(kvq, "plain", 2, 2, T, 4, 512)
    n = 20
    q, dk, dv = tree_inputs(9, 2, n, 2, 3)
    mask = tree_mask(2, 2, n=n)
    mask[:, 4:9] = False
    mask[1] = False
    tree_check(q, dk, dv, mask, ks, vs, cache.tree_attn(0, q, dk, dv, mask.cuda()))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [0, 200])
@pytest.mark.parametrize("n,real,G", [(14, 9, 5), (8, 3, 1), (7, 2, 1)])
def test_tree_padding_never_leaks(kvq, dtype, T, n, real, G):
    """Padded nodes hold NaN, infinities and the type's extremes; no other node's output notices."""
    cache, _, ks, vs = make_cache(kvq, "plain", 1, 2, T, 4, 512)
    q, dk, dv = tree_inputs(11, 1, n, 2, G, dtype)
    mask = torch.zeros(n, n, dtype=torch.bool)
    mask[:real, :real] = tree_mask(3, n=real)
    want = cache.tree_attn(0, q, dk, dv, mask.cuda())
    big = torch.finfo(dtype).max
    for x in (dk, dv):
        for i, bad in enumerate((math.nan, math.inf, -math.inf, big, -big)):
            x[:, real + i] = bad
    q[:, real:] = math.nan
    q[:, real + 1] = math.inf
    got = cache.tree_attn(0, q, dk, dv, mask.cuda())
    assert torch.equal(got[:, :real], want[:, :real])


def test_tree_strided_inputs(kvq):
    """q, k, v as slices of one projection; an output and a scale of the caller's."""
    cache, _, ks, vs = make_cache(kvq, "plain", 2, 2, 500, 2, 512)
    qkv = randn(13, 2, 6, 3 * 2 + 2 + 2, 128)
    q, dk, dv = qkv[:, :, :6], qkv[:, :, 6:8], qkv[:, :, 8:]
    out = torch.zeros(2, 6, 6, 128, dtype=BF, device="cuda")
    assert cache.tree_attn(0, q, dk, dv, sm_scale=0.2, out=out) is out
    tree_check(q, dk, dv, None, ks, vs, out, 0.2)
    tree_check(q, dk, dv, None, ks, vs, cache.tree_attn(0, q, dk, dv, sm_scale=-0.05), -0.05)


def test_tree_equals_decode_of_one_token(kvq):
    """A tree of one node equals appending its token at 16 bits and decoding."""
    cache, _, ks, vs = make_cache(kvq, "plain", 2, 2, 300, 16, 512)
    q, dk, dv = tree_inputs(17, 2, 1, 2, 4)
    tree = cache.tree_attn(0, q, dk, dv)
    dec = cache.append_decode(0, dk, dv, q[:, 0].contiguous())
    assert ((tree[:, 0].float() - dec).abs() <= 2 * UBF * dec.abs() + 0.01 * dec.abs().amax(-1, keepdim=True)).all()


@pytest.mark.parametrize("n,G", [(9, 7), (1, 7), (2, 4)])
def test_tree_streams_and_graphs(kvq, n, G):
    """Two calls at once on two streams, and two captured graphs replayed in turn and together."""
    cache, _, ks, vs = make_cache(kvq, "plain", 2, 2, 3000, 2, 4096)
    a, b = tree_inputs(19, 2, n, 2, G), tree_inputs(23, 2, n, 2, G)
    wa, wb = cache.tree_attn(0, *a), cache.tree_attn(0, *b)
    tree_check(*a, None, ks, vs, wa)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(cache.tree_attn(0, *a, stream=s1), cache.tree_attn(0, *b, stream=s2)) for _ in range(20)]
    torch.cuda.synchronize()
    for x, y in got:
        assert torch.equal(x, wa) and torch.equal(y, wb)
    oa, ob = torch.zeros_like(wa), torch.zeros_like(wb)
    ga, gb = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(ga):
        cache.tree_attn(0, *a, out=oa)
    with torch.cuda.graph(gb):
        cache.tree_attn(0, *b, out=ob)
    for _ in range(5):
        oa.zero_()
        ob.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            ga.replay()
        with torch.cuda.stream(s2):
            gb.replay()
        torch.cuda.synchronize()
        assert torch.equal(oa, wa) and torch.equal(ob, wb)
    cache.device_status()


def test_tree_python_refusals(kvq):
    cache, _, _, _ = make_cache(kvq, "plain", 2, 2, 100, 4, 512)
    q, dk, dv = tree_inputs(29, 2, 4, 2, 3)
    m = torch.ones(4, 4, dtype=torch.bool, device="cuda")
    for bad in (lambda: cache.tree_attn(0, q[:1], dk, dv), lambda: cache.tree_attn(0, q, dk[:, :3], dv),
                lambda: cache.tree_attn(0, q, dk, dv[:, :, :1]), lambda: cache.tree_attn(0, q, dk, dv, m[:3]),
                lambda: cache.tree_attn(0, q, dk, dv, m.float()), lambda: cache.tree_attn(0, q, dk, dv, m.cpu()),
                lambda: cache.tree_attn(0, q, dk, dv, out=q[:, :2]), lambda: cache.tree_attn(0, q.cpu(), dk, dv),
                lambda: cache.tree_attn(0, q, dk, dv, torch.ones(4, 8, dtype=torch.bool, device="cuda")[:, ::2])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: cache.tree_attn(0, q.float(), dk, dv), lambda: cache.tree_attn(0, q, dk, dv.float()),
                lambda: cache.tree_attn(0, q, dk.half(), dv.half())):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: cache.tree_attn(1, q, dk, dv), lambda: cache.tree_attn(0, q[:, :, :5], dk, dv),
                lambda: cache.tree_attn(0, q, dk, dv, sm_scale=math.inf)):
        with pytest.raises((kvq.KVQError, ValueError)):
            bad()


# ---------------------------------------------------------- used together

@pytest.mark.parametrize("mode", MODES)
def test_draft_verify_commit_read(kvq, mode):
    """One round of drafting: rotate the projection's q and k, attend the tree over the cache, append the accepted
    path's Keys and Values, read the cache back; then the same for the next round on the grown cache."""
    B, H, G, n = 2, 2, 4, 6
    T = 400
    cache, scale, ks, vs = make_cache(kvq, mode, B, H, T, 4, 1024)
    rope = kvq.Rope(128, scaling="linear", factor=2.0)
    for r in range(3):
        qkv = randn(31 + r, B, n, H * G + 2 * H, 128)
        depth = torch.tensor([0, 1, 1, 2, 2, 3], device="cuda")
        seen = torch.zeros(n, n, dtype=torch.bool)
        for i, p in enumerate([-1, 0, 0, 1, 2, 3]):
            if p >= 0:
                seen[i] = seen[p]
            seen[i, i] = True
        q, k = kvq.kvq_rope(rope, T + depth, qkv[:, :, :H * G], qkv[:, :, H * G:H * G + H])
        rope_check(rope, (T + depth).expand(B, n), qkv[:, :, :H * G], q)
        v = qkv[:, :, H * G + H:]
        out = cache.tree_attn(0, q, k, v, seen.cuda())
        tree_check(q, k, v, seen, ks, vs, out)
        path = torch.tensor([0, 1, 3, 5], device="cuda")
        cache.append(0, k[:, path].contiguous(), v[:, path].contiguous())
        T += 4
        ks, vs = held(kvq, cache, mode, B, H, T, scale)
        rk, rv = cache.read(0, T - 4, 4, dtype=F32)
        assert torch.equal(rk.cpu().transpose(1, 2), ks[:, :, -4:]) and torch.equal(rv.cpu().transpose(1, 2), vs[:, :, -4:])
        # what was appended comes back within half a step of its width (16 bits in the window and the staged block)
        x = k[:, path].float() / scale.cuda()
        bits = cache.query(0)["bits"] if mode == "plain" else 16
        step = (x.amax(-1) - x.amin(-1)) * 1.002 / (2 ** bits - 1)  # the range is rounded up to binary16
        worst = ((rk - k[:, path].float()).abs() / scale.cuda()).amax(-1)
        assert (worst <= 0.5 * step + 2.0 ** -20 * x.abs().amax(-1)).all()


def test_first_calls_in_a_capture():
    """A fresh process whose first calls of the operators are captured, on a cache that nothing has touched yet."""
    code = r"""
import torch
import mixed_precision_kv_kvq_b200 as kvq
torch.cuda.init()
cache = kvq.KVQCache(1, 1, 2, 512 * 2 * 2 * (16 * 4 + 4), [4])
q = torch.randn(1, 9, 8, 128, device="cuda").bfloat16()
k, v = torch.randn(1, 9, 2, 128, device="cuda").bfloat16(), torch.randn(1, 9, 2, 128, device="cuda").bfloat16()
pos = torch.arange(9, device="cuda")
rope = kvq.Rope(128)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    a, b = kvq.kvq_rope(rope, pos, q, k)
    out = cache.tree_attn(0, a, b, v)
cache.device_status()
graph.replay()
torch.cuda.synchronize()
cache.device_status()
a2, b2 = kvq.kvq_rope(rope, pos, q, k)
assert torch.equal(a, a2) and torch.equal(b, b2) and torch.equal(out, cache.tree_attn(0, a2, b2, v))
assert torch.equal(out[:, 0], v[:, 0].repeat_interleave(4, 1))
cache.append(0, b, v)
graph2 = torch.cuda.CUDAGraph()
rk = torch.empty_like(k)
with torch.cuda.graph(graph2):
    cache.read(0, 0, 9, k_out=rk)
graph2.replay()
torch.cuda.synchronize()
assert torch.equal(rk, cache.read(0)[0])
print("ok")
"""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("ok"), r.stderr[-2000:]


@pytest.mark.parametrize("n,G", [(2, 2), (12, 4)])
def test_tree_extremes_that_are_seen_stay_finite(kvq, n, G):
    """Drafted values at and beyond binary16's range, and queries of a tiny and a huge row, in nodes that see them."""
    cache, _, ks, vs = make_cache(kvq, "plain", 1, 2, 200, 4, 512)
    q, dk, dv = tree_inputs(37, 1, n, 2, G, F32)
    dk[:, 0, :, :5] = torch.tensor([math.inf, -math.inf, 1e30, -1e30, math.nan], device="cuda")
    dv[:, 0, :, :5] = torch.tensor([math.inf, -math.inf, 1e30, -1e30, math.nan], device="cuda")
    q[:, 1] *= 1e-6
    out = cache.tree_attn(0, q, dk, dv)
    assert torch.isfinite(out).all()
    # a node that sees the first one not at all is as if it were ordinary
    mask = torch.ones(n, n, dtype=torch.bool).tril()
    mask[1:, 0] = False
    good_k, good_v = dk.clone(), dv.clone()
    good_k[:, 0] = good_v[:, 0] = 0.5
    tree_check(q[:, 1:], good_k[:, 1:], good_v[:, 1:], mask[1:, 1:], ks, vs, cache.tree_attn(0, q, dk, dv, mask.cuda())[:, 1:])


@pytest.mark.parametrize("R,Z", [(0.0, 3.0), (1e-3, 8.0), (30.0, -15.0), (2.0, 60000.0)])
def test_tree_keys_with_offsets(kvq, R, Z):
    """Groups that are constant, nearly constant beside a large zero, or wide: the range's floor in the score's centre."""
    B, H, T = 1, 1, 300
    for fbit in (2, 8):
        cache = kvq.KVQCache(1, B, H, 512 * B * H * 2 * (16 * fbit + 4), [fbit])
        g = torch.Generator().manual_seed(1)
        k = Z + R * torch.rand(B, T, H, 128, generator=g)
        v = torch.randn(B, T, H, 128, generator=g)
        cache.append(0, k.cuda(), v.cuda())
        ks, vs = held(kvq, cache, "plain", B, H, T, None)
        q, dk, dv = tree_inputs(3, B, 6, H, 3)
        q *= 0.2 if abs(Z) < 100 else 1e-4
        tree_check(q, dk, dv, None, ks, vs, cache.tree_attn(0, q, dk, dv))


@pytest.mark.parametrize("n,G", [(1, 4), (16, 4)])
def test_raw_stream_handles_own_what_the_call_allocates(kvq, n, G):
    """A stream given as its handle: the workspace and the output are not the current stream's to hand out meanwhile."""
    cache, *_ = make_cache(kvq, "plain", 2, 2, 500, 4, 1024)
    q, dk, dv = tree_inputs(21, 2, n, 2, G)
    rope, pos = kvq.Rope(128), torch.arange(n, device="cuda")
    want, turned, (rk, rv) = cache.tree_attn(0, q, dk, dv), kvq.kvq_rope(rope, pos, q, dk), cache.read(0)
    nbytes = kvq.kvq_tree_workspace(cache.handle, 0, 2 * G, n)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    h = side.cuda_stream
    out, got, back = cache.tree_attn(0, q, dk, dv, stream=h), kvq.kvq_rope(rope, pos, q, dk, stream=h), cache.read(0, stream=h)
    junk = [torch.full((size,), 0x7F, dtype=torch.uint8, device="cuda") for size in (nbytes, out.numel() * 2) for _ in range(4)]
    side.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all(torch.equal(a, b) for a, b in zip(got + back, turned + (rk, rv)))
    assert all(bool((j == 0x7F).all()) for j in junk)
    # the default stream's handle
    assert torch.equal(cache.tree_attn(0, q, dk, dv, stream=torch.cuda.default_stream().cuda_stream), want)


@pytest.mark.parametrize("T", [0, 130])
@pytest.mark.parametrize("n,G", [(300, 2), (60, 1), (30, 1), (12, 1)])
def test_tree_low_scores_seen_late(kvq, T, n, G):
    """Scores far below zero (2^-60 against no maximum), some rows' first tokens in the last drafted tile, one row's nowhere."""
    B, H = 1, 2
    cache = kvq.KVQCache(1, B, H, 512 * B * H * 2 * (16 * 8 + 4), [8])
    g = torch.Generator().manual_seed(3)
    k, v = 0.1 * torch.randn(B, max(T, 1), H, 128, generator=g), torch.randn(B, max(T, 1), H, 128, generator=g)
    k[..., 0] = -22.0
    if T:
        cache.append(0, k.cuda(), v.cuda())
    ks, vs = held(kvq, cache, "plain", B, H, T, None)
    q, dk, dv = tree_inputs(5, B, n, H, G)
    q *= 0.1
    dk *= 0.1
    q[..., 0] = 22.0
    dk[..., 0] = -22.0
    late = 128 if n > 128 else n // 2
    mask = torch.ones(n, n, dtype=torch.bool)
    mask[::2, :late] = False
    mask[1::4, late:] = False
    mask[5] = False
    tree_check(q, dk, dv, mask, ks, vs, cache.tree_attn(0, q, dk, dv, mask.cuda()))
