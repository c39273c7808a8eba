"""Cases of the rotary, tree-attention and read-back operators.

Shapes are those of this repository's decode workloads: 4 KV / 28 query heads
(7B), 8 / 40 (32B), 8 / 64 (Llama-70B), 2 / 4 (tiny); 32K contexts, blocks at
2, 4, 8 or 16 bits.  Keys carry outlier channels and a migration factor, as
the cache expects them.  The cache's contents follow the method's definition:
a token is quantized per head over its 128 channels at the width its block
has when it arrives, and shrinks with the block (16 -> 8 -> 4 -> 2).
"""
import math

import torch

own = False

D = 128
BF16, F32 = "bf16", "f32"
DTYPES = {BF16: torch.bfloat16, F32: torch.float32}


def listed():
    return [
        # a drafted tree of a small model on a short context: the call's latency counts
        {"name": "tree tiny n4 1100", "op": "tree", "batch": 1, "kv_heads": 2, "group": 2, "nodes": 4, "tokens": 1100,
         "fbit": 4, "mask": "tree"},
        # the plain decode step as a tree of one node: one token a sequence, bound by the cache's bytes
        {"name": "tree 7b n1 32k 4bit", "op": "tree", "batch": 16, "kv_heads": 4, "group": 7, "nodes": 1,
         "tokens": 32701, "fbit": 4, "mask": "chain"},
        # verifying a tree of 16 drafted tokens a sequence on a long 2-bit context
        {"name": "tree 7b n16 32k 2bit", "op": "tree", "batch": 16, "kv_heads": 4, "group": 7, "nodes": 16,
         "tokens": 32768, "fbit": 2, "mask": "tree"},
        # a wide tree, odd in every size, on an 8-bit block: bound by the products and the exponentials
        {"name": "tree 70b n63 16k 8bit", "op": "tree", "batch": 8, "kv_heads": 8, "group": 8, "nodes": 63,
         "tokens": 16383, "fbit": 8, "mask": "tree"},
        # a short chain of drafted tokens on a block that still holds 16 bits
        {"name": "tree 32b n5 5k 16bit", "op": "tree", "batch": 4, "kv_heads": 8, "group": 5, "nodes": 5,
         "tokens": 4999, "fbit": 16, "mask": "chain"},
        # the latest tokens of one sequence read back
        {"name": "read tiny 100", "op": "read", "batch": 1, "kv_heads": 2, "tokens": 1100, "fbit": 4, "start": 1000,
         "count": 100, "dtype": BF16},
        # a whole 2-bit block read back for another engine
        {"name": "read 7b 32k 2bit", "op": "read", "batch": 16, "kv_heads": 4, "tokens": 32768, "fbit": 2, "start": 0,
         "count": 32768, "dtype": BF16},
        # an odd range of a 4-bit block in fp32, to be quantized again elsewhere
        {"name": "read 70b 9001 4bit f32", "op": "read", "batch": 8, "kv_heads": 8, "tokens": 16000, "fbit": 4,
         "start": 1357, "count": 9001, "dtype": F32},
        # one decode step's queries and Keys
        {"name": "rope 7b decode", "op": "rope", "batch": 16, "tokens": 1, "q_heads": 28, "kv_heads": 4, "rot_dim": 128,
         "layout": "half", "scaling": "none", "factor": 1.0, "first": 32768, "dtype": BF16},
        # a chunk of a prompt far beyond the trained length
        {"name": "rope 70b chunk yarn", "op": "rope", "batch": 8, "tokens": 4096, "q_heads": 64, "kv_heads": 8,
         "rot_dim": 128, "layout": "half", "scaling": "yarn", "factor": 16.0, "first": 100000, "dtype": BF16},
        # part of the head, neighbouring pairs, an odd number of tokens, fp32
        {"name": "rope part 1001 f32", "op": "rope", "batch": 3, "tokens": 1001, "q_heads": 40, "kv_heads": 8,
         "rot_dim": 64, "layout": "interleaved", "scaling": "linear", "factor": 4.0, "first": 7, "dtype": F32},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))) - 0.5))))


def draw(rng):
    op = rng.choice(["tree", "tree", "read", "rope"])
    while True:
        kv_heads = rng.randint(1, 8)
        if op == "rope":
            case = {"op": op, "batch": _log(rng, 1, 16), "tokens": _log(rng, 1, 4096), "q_heads": kv_heads * rng.randint(1, 8),
                    "kv_heads": kv_heads, "rot_dim": rng.choice([32, 48, 64, 96, 128, 128]),
                    "layout": rng.choice(["half", "interleaved"]), "scaling": rng.choice(["none", "linear", "ntk", "yarn"]),
                    "factor": rng.choice([2.0, 4.0, 16.0]), "first": _log(rng, 1, 1000000), "dtype": rng.choice([BF16, BF16, F32])}
            if case["scaling"] == "none":
                case["factor"] = 1.0
        else:
            case = {"op": op, "batch": _log(rng, 1, 16), "kv_heads": kv_heads, "tokens": _log(rng, 1, 32768),
                    "fbit": rng.choice([2, 2, 4, 4, 8, 16])}
            if op == "tree":
                case.update(group=rng.randint(1, 8), nodes=_log(rng, 1, 96), mask=rng.choice(["tree", "tree", "shared", "chain"]))
            else:
                case["start"] = rng.randint(0, case["tokens"] - 1)
                case["count"] = rng.randint(1, case["tokens"] - case["start"])
                case["dtype"] = rng.choice([BF16, BF16, F32])
        w = work(case)
        if w["bytes"] <= 1.1e9 and w["flops"] <= 2.7e11:
            return case


# ------------------------------------------------------------------ inputs

def _keys_values(gen, batch, tokens, heads):
    k = torch.randn(batch, tokens, heads, D, generator=gen, device="cuda", dtype=torch.float32)
    v = torch.randn(batch, tokens, heads, D, generator=gen, device="cuda", dtype=torch.float32)
    loud = torch.randint(0, D, (heads, 2), generator=gen, device="cuda")
    k.mul_(1.0 + 19.0 * torch.zeros(heads, D, device="cuda").scatter_(1, loud, 1.0))
    return k.bfloat16(), v.bfloat16()


def _lambda(k):
    return k[0, :512].float().abs().amax(0).sqrt().clamp_min(0.05)  # [heads][128]


def _capacity(case):
    return -(-case["tokens"] // 512) * 512  # tokens the block holds at its final width


def _toward(x, up):
    """fp32 -> binary16 rounded down (up: rounded up): the nearest one, moved a step where it lies on the wrong side."""
    h = x.half() + 0.0  # no -0
    wrong = h.float() < x if up else h.float() > x
    i = h.view(torch.int16)
    i = i ^ ((i >> 15) & 0x7FFF)  # in the order of the values
    i = torch.where(wrong, i + 1 if up else i - 1 - (i == 0).to(torch.int16), i)
    return (i ^ ((i >> 15) & 0x7FFF)).view(torch.float16)


def _quantize(x, bits):
    """Codes, range and zero of groups along the last axis, every step rounded to fp32 on its own."""
    z = _toward(x.amin(-1, keepdim=True), False)
    r = _toward(x.amax(-1, keepdim=True) - z.float(), True)
    top = torch.full((1,), float(2 ** bits - 1), device=x.device)
    inv = torch.where(r > 0, top / r.float(), torch.zeros_like(top))
    c = (x - z.float()).mul_(inv).add_(0.5).floor_().clamp_(0, 2 ** bits - 1).to(torch.int64 if bits == 16 else torch.int32)
    return c, r, z


def _shrink(c, bits):
    """One level of the Equivalent Right Shift, 2 bits -> bits."""
    return ((4 ** bits - 2 ** bits + 1) * (c + 2 ** (bits - 1))) >> (3 * bits)


def _blocks(x, fbit, capacity):
    """What the cache holds of x [b][t][h][128] (fp32): codes [b][h][t][128] at the block's width, range, zero, width."""
    tokens, x = x.shape[1], x.transpose(1, 2)
    widths = [b for b in (16, 8, 4, 2) if b >= fbit]
    ends = [capacity * fbit // b for b in widths]
    last = next(i for i, e in enumerate(ends) if tokens <= e)
    codes, ranges, zeros = [], [], []
    for e in range(last + 1):
        part = x[:, :, 0 if e == 0 else ends[e - 1]:min(ends[e], tokens)]
        c, r, z = _quantize(part, widths[e])
        for b in widths[e + 1:last + 1]:
            c = _shrink(c, b)
        codes.append(c.to(torch.uint8 if widths[last] <= 8 else torch.int32))
        ranges.append(r)
        zeros.append(z)
    return torch.cat(codes, 2), torch.cat(ranges, 2), torch.cat(zeros, 2), widths[last]


def _cache(case, gen):
    """The block's contents: the framework's cache, or the codes of the definition."""
    k, v = _keys_values(gen, case["batch"], case["tokens"], case["kv_heads"])
    lam = _lambda(k)
    if own:
        import mixed_precision_kv_kvq_b200 as kvq

        per_token = case["batch"] * case["kv_heads"] * 2 * (16 * case["fbit"] + 4)
        cache = kvq.KVQCache(1, case["batch"], case["kv_heads"], _capacity(case) * per_token, [case["fbit"]])
        cache.set_lambda(0, lam)
        cache.append(0, k, v)
        return {"cache": cache}
    inv = (1.0 / lam.double()).float()
    kc, kr, kz, bits = _blocks(k.float().mul_(inv), case["fbit"], _capacity(case))
    vc, vr, vz, _ = _blocks(v.float(), case["fbit"], _capacity(case))
    return {"k": (kc, kr, kz), "v": (vc, vr, vz), "bits": bits, "lam": lam}


def _tree_mask(gen, batch, nodes):
    """visible[b][i][j]: j is i or one of its ancestors; every node hangs from an earlier one or from the context."""
    seen = torch.zeros(batch, nodes, nodes, dtype=torch.bool, device="cuda")
    u = torch.rand(batch, nodes, generator=gen, device="cuda")
    at = torch.arange(batch, device="cuda")
    for i in range(nodes):
        parent = (u[:, i] * (i + 1)).long() - 1  # -1: the context
        seen[:, i] = seen[at, parent.clamp_min(0)] & (parent >= 0)[:, None]
        seen[:, i, i] = True
    return seen


def _inv_freq(case):
    """Angle per position of each pair, and what cos and sin are multiplied by."""
    d, theta, f = case["rot_dim"], 10000.0, case["factor"]
    i = torch.arange(0, d, 2, dtype=torch.float64)
    if case["scaling"] == "ntk":
        theta *= f ** (d / (d - 2))
    inv, mag = theta ** (-i / d), 1.0
    if case["scaling"] == "linear":
        inv = inv / f
    if case["scaling"] == "yarn":  # between interpolated (slow) and unchanged (fast) pairs over a context of 4096
        turns = lambda n: d * math.log(4096 / (n * 2 * math.pi)) / (2 * math.log(theta))  # noqa: E731
        low, high = max(math.floor(turns(32.0)), 0), min(math.ceil(turns(1.0)), d - 1)
        ramp = ((i / 2 - low) / max(high - low, 0.001)).clamp(0, 1)
        inv, mag = inv / f * ramp + inv * (1 - ramp), 0.1 * math.log(f) + 1.0
    return inv, mag


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "rope":
        heads = case["q_heads"] + 2 * case["kv_heads"]
        qkv = torch.randn(case["batch"], case["tokens"], heads, D, generator=gen, device="cuda").to(DTYPES[case["dtype"]])
        at = torch.randint(0, case["first"], (case["batch"], 1), generator=gen, device="cuda")
        state = {"op": "rope", "q": qkv[:, :, :case["q_heads"]], "k": qkv[:, :, case["q_heads"]:case["q_heads"] + case["kv_heads"]],
                 "pos": at + torch.arange(case["tokens"], device="cuda")}
        if own:
            import mixed_precision_kv_kvq_b200 as kvq

            state["rope"] = kvq.Rope(case["rot_dim"], layout=case["layout"], scaling=case["scaling"], factor=case["factor"],
                                     original_tokens=4096)
        else:
            inv, mag = _inv_freq(case)
            state.update(inv=inv.cuda(), mag=mag, layout=case["layout"])
        return state
    state = {"op": case["op"], **_cache(case, gen)}
    if case["op"] == "read":
        state.update(start=case["start"], count=case["count"], dtype=DTYPES[case["dtype"]])
        return state
    b, h, n = case["batch"], case["kv_heads"], case["nodes"]
    state["q"] = torch.randn(b, n, h * case["group"], D, generator=gen, device="cuda").bfloat16()
    state["dk"], state["dv"] = _keys_values(gen, b, n, h)
    state["mask"] = None
    if case["mask"] != "chain":
        mask = _tree_mask(gen, b if case["mask"] == "tree" else 1, n)
        state["mask"] = mask if case["mask"] == "tree" else mask[0]
    return state


# --------------------------------------------------------------------- run

def _dequantized(group, bits):
    c, r, z = group
    return c.float().mul_(r.float() / torch.full((1,), float(2 ** bits - 1), device=r.device)).add_(z.float())


def _rope_plain(x, s):
    half = s["inv"].numel()
    angle = s["pos"][:, :, None, None].double() * s["inv"]
    cos, sin = (angle.cos() * s["mag"]).float(), (angle.sin() * s["mag"]).float()
    y = x.float()
    if s["layout"] == "half":
        a, b = y[..., :half], y[..., half:2 * half]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0:2 * half:2], y[..., 1:2 * half:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, y[..., 2 * half:]], -1).to(x.dtype)


def _tree_plain(s):
    b, n, hq, _ = s["q"].shape
    h = s["dk"].shape[2]
    scale = D ** -0.5
    rows = lambda x: x.view(b, n, h, hq // h, D).permute(0, 2, 1, 3, 4).reshape(b, h, n * (hq // h), D)  # noqa: E731
    q = s["q"].float()
    moved = (q.view(b, n, h, hq // h, D) * s["lam"][:, None, :]).view(b, n, hq, D)
    far = rows(moved) @ _dequantized(s["k"], s["bits"]).transpose(-1, -2)
    near = rows(q) @ s["dk"].float().permute(0, 2, 3, 1)
    mask = s["mask"]
    if mask is None:
        mask = torch.ones(n, n, dtype=torch.bool, device=q.device).tril_()
    mask = mask.expand(b, n, n).repeat_interleave(hq // h, 1)[:, None]
    near = torch.where(mask, near, torch.full((), -math.inf, device=q.device))
    top = torch.maximum(far.amax(-1, keepdim=True), near.amax(-1, keepdim=True)) * scale
    far, near = far.mul_(scale).sub_(top).exp_(), near.mul_(scale).sub_(top).exp_()
    total = far.sum(-1, keepdim=True) + near.sum(-1, keepdim=True)
    out = (far @ _dequantized(s["v"], s["bits"]) + near @ s["dv"].float().transpose(1, 2)) / total
    return out.view(b, h, n, hq // h, D).permute(0, 2, 1, 3, 4).reshape(b, n, hq, D).bfloat16()


def run(s):
    if s["op"] == "rope":
        if own:
            import mixed_precision_kv_kvq_b200 as kvq

            return kvq.kvq_rope(s["rope"], s["pos"], s["q"], s["k"])
        return _rope_plain(s["q"], s), _rope_plain(s["k"], s)
    if s["op"] == "read":
        if own:
            return s["cache"].read(0, s["start"], s["count"], dtype=s["dtype"])
        part = lambda g: tuple(x[:, :, s["start"]:s["start"] + s["count"]] for x in g)  # noqa: E731
        k = (_dequantized(part(s["k"]), s["bits"]) * s["lam"][:, None, :]).to(s["dtype"])
        v = _dequantized(part(s["v"]), s["bits"]).to(s["dtype"])
        return k.transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous()
    if own:
        return s["cache"].tree_attn(0, s["q"], s["dk"], s["dv"], s["mask"])
    return _tree_plain(s)


# ------------------------------------------------------------- work, exact

def _bits_now(case):
    return next(b for b in (16, 8, 4, 2) if b >= case["fbit"] and case["tokens"] <= _capacity(case) * case["fbit"] // b)


def work(case):
    size = 2 if case.get("dtype", BF16) == BF16 else 4
    if case["op"] == "rope":
        values = case["batch"] * case["tokens"] * (case["q_heads"] + case["kv_heads"]) * D
        return {"bytes": 2 * values * size + 8 * case["batch"] * case["tokens"], "flops": 3 * values * case["rot_dim"] // D}
    streams, per_token = case["batch"] * case["kv_heads"], 2 * (16 * _bits_now(case) + 4)
    if case["op"] == "read":
        n = streams * case["count"]
        return {"bytes": n * (per_token + 2 * D * size), "flops": 5 * n * D}
    n, rows = case["nodes"], case["nodes"] * case["group"]
    masks = {"tree": case["batch"], "shared": 1, "chain": 0}[case["mask"]]
    return {"bytes": streams * (case["tokens"] * per_token + 2 * rows * D * 2 + 2 * n * D * 2) + masks * n * n,
            "flops": 4 * D * streams * rows * (case["tokens"] + n)}


def _exact_values(group, bits, b, h):
    c, r, z = (x[b, h].double() for x in group)
    return z + c * r / (2.0 ** bits - 1.0)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        outs = []
        for x in (s["q"], s["k"]):
            y = x.double().clone()
            for p in range(case["rot_dim"] // 2):
                i, j = (p, p + case["rot_dim"] // 2) if case["layout"] == "half" else (2 * p, 2 * p + 1)
                turn = torch.polar(torch.full_like(s["pos"], s["mag"], dtype=torch.float64), s["pos"].double() * s["inv"][p])
                z = torch.complex(x[..., i].double(), x[..., j].double()) * turn[:, :, None]
                y[..., i], y[..., j] = z.real, z.imag
            outs.append(y)
        return tuple(outs)
    streams = [(b, h) for b in range(case["batch"]) for h in range(case["kv_heads"])]
    if case["op"] == "read":
        at = slice(case["start"], case["start"] + case["count"])
        k = torch.empty(case["batch"], case["count"], case["kv_heads"], D, dtype=torch.float64, device="cuda")
        v = torch.empty_like(k)
        for b, h in streams:
            k[b, :, h] = (_exact_values(s["k"], s["bits"], b, h) * s["lam"][h].double())[at]
            v[b, :, h] = _exact_values(s["v"], s["bits"], b, h)[at]
        return k, v
    g, n = case["group"], case["nodes"]
    out = torch.empty(case["batch"], n, case["kv_heads"] * g, D, dtype=torch.float64, device="cuda")
    ban = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1) if s["mask"] is None else ~s["mask"]
    for b, h in streams:
        keys = torch.cat([_exact_values(s["k"], s["bits"], b, h) * s["lam"][h].double(), s["dk"][b, :, h].double()])
        values = torch.cat([_exact_values(s["v"], s["bits"], b, h), s["dv"][b, :, h].double()])
        hidden = torch.cat([torch.zeros(n, case["tokens"], dtype=torch.bool, device="cuda"), ban[b] if ban.dim() == 3 else ban], 1)
        for i in range(g):
            score = (s["q"][b, :, h * g + i].double() @ keys.T) / math.sqrt(D)
            out[b, :, h * g + i] = torch.softmax(score.masked_fill(hidden, -math.inf), -1) @ values
    return out
