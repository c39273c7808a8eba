"""How far tree attention's output may be off in the root mean square, and what
an output that lost or doubled tokens would look like.

A rounding to type t is off by at most half a step, u_t = finfo(t).eps / 2 relative
to the value (bf16 2^-8, fp16 2^-11).  Roundings of different values are
independent, so their squares add.  Below every one counts with its full
half step, though a value's error is spread evenly over the half step and so has
1 / sqrt(3) of it in the root mean square: that factor is the slack for how evenly.
With w the weights, o the row's output and s the scale:
 * the output is rounded to bf16: u_bf o.
 * wide path (more than 8 rows n G): p is rounded (u w v, and 2^-25 v below 2^-14
   of a largest p of about 1), a cached Value goes through its group's centre c
   (u c, then u v; a 16-bit code and, in a block of another width, its range u (v - c)
   each), a drafted Value is rounded once (u v).
 * the query is rounded once, the same for every token: of channel i by u q_i,
   which moves the output by s u q_i sum_t w_t k_ti (v_t - o).
 * Keys: codes of 8 bits and fewer are exact; 16-bit ones are rounded, u (k - c) each;
   per-channel groups go in as values, u k each and their centres u c, the same
   for every token of a block; drafted ones u k.  A Key moves the output by
   w_t (v_t - o) times its score's error.
 * fp32: sums of |q_i k_i| by 2^-20, the centre's part (a 22-bit pair) by 2^-21, the
   maximum's subtraction and the exponential by 2^-22 (|score| + 1), each token its own.
 * path of up to 8 rows: the query in 2^-16 of its largest channel (times lambda),
   Key codes exact, drafted tokens fp32; p R rounded, u (|v| + |c|) w; and
   Value codes that enter the product as subnormals, off by up to 2^-12 of
   sum_t w_t R_t altogether: that one is added whole.
The root mean square over a stream (n G rows of 128 channels) must be within 1.25
times, over one row within 2.5 times this sum: over a row the errors are as few as
its channels or its loudest query channels, so it scatters more (2.5 sqrt(3) is 4.3
deviations of a sum of evenly spread errors, 1.25 sqrt(3) is 2.2 of an average over
a thousand)."""
import math

import torch

U16, UBF = 2.0 ** -11, 2.0 ** -8


def sees(mask, B, n):
    m = torch.ones(n, n, dtype=torch.bool).tril() if mask is None else mask.bool()
    return m.expand(B, n, n)


class Stream:
    """One (sequence, KV head) stream's tokens, cached ones before drafted ones, in fp64, and how each is rounded."""

    def __init__(self, ks, vs, dk, dv, mode, bits, lam, narrow, cancel=False):
        """ks, vs [T][128] with .centre, .range; dk, dv [n][128]; lam [128] or None.  cancel: every query's channels cancel
        exactly (sums of equal powers of two, rounded nowhere), so that a cached Key's centre adds no error to a score, and the
        groups' ranges are small beside their zeros, so that a Key's distance from its centre is rounded, u (k - c)."""
        dev = dk.device
        T, n = ks.shape[0], dk.shape[0]
        d = lambda x: x.to(dev).double()  # noqa: E731
        zero = torch.zeros(n, 128, dtype=torch.float64, device=dev)
        self.T, self.n, self.narrow = T, n, narrow
        dk, dv = (torch.nan_to_num(d(x), 0, 0, 0) for x in (dk, dv))  # what is not seen may be anything
        self.k, self.v = torch.cat([d(ks), dk]), torch.cat([d(vs), dv])
        self.kc = torch.cat([d(ks.centre).expand(T, 128), zero])
        vc = torch.cat([d(vs.centre).expand(T, 128), zero])
        self.vr = torch.cat([d(vs.range), zero[:, :1]])
        self.lam = torch.ones(128, dtype=torch.float64, device=dev) if lam is None else d(lam)
        at = torch.arange(T + n, device=dev)
        cached = at < T
        if mode == "window":
            code16 = (at == 0) | (at >= T - 128)
        elif mode == "channel":
            code16 = at >= T - T % 128
        else:
            code16 = torch.zeros_like(cached)
        code16 = ((code16 | (bits == 16)) & cached)[:, None]
        chan = (cached[:, None] & ~(at >= T - T % 128)[:, None]) if mode == "channel" else torch.zeros_like(code16)
        drafted = ~cached[:, None]
        away = (self.k - self.kc).abs()
        self.size = torch.where(cached[:, None], away, self.k.abs()) if cancel else self.k.abs()
        self.kerr = U16 * torch.where(chan | drafted, self.k.abs(), torch.where(code16, away, 0.0))
        self.kblock = U16 * torch.where(chan, self.kc.abs(), 0.0)
        self.blocks = (T - T % 128) // 128 if mode == "channel" else 0
        v2, c2 = self.v ** 2, vc ** 2
        self.verr2 = U16 ** 2 * (2 * v2 + c2 + torch.where(code16, 2 * (self.v - vc) ** 2, 0.0))  # p's rounding and the Value's own
        if cancel:
            self.kerr = torch.where(cached[:, None], U16 * away * (1 + code16), self.kerr)
        if narrow:
            self.kerr.zero_()
            self.kblock.zero_()
            self.verr2 = torch.where(cached[:, None], U16 ** 2 * (self.v.abs() + vc.abs()) ** 2, 0.0)
            self.verr2 = self.verr2 + U16 ** 2 * v2 * cached[:, None]

    def weights(self, q, seen, sm_scale):
        vis = torch.cat([torch.ones(self.n, self.T, dtype=torch.bool, device=q.device), seen], 1)
        s = torch.where(vis, sm_scale * (q @ self.k.T), torch.full((), -math.inf, dtype=torch.float64, device=q.device))
        top = s.amax(1, keepdim=True)
        p = torch.where(vis, torch.exp(s - torch.where(top.isfinite(), top, 0.0)), 0.0)
        total = p.sum(1, keepdim=True)
        return torch.where(total > 0, p / total, 0.0), s, total.clamp_min(1.0), vis

    def expect(self, q, seen, sm_scale):
        """q [n][128] of one query head -> output [n][128] and the square it may be off by."""
        w, s, total, vis = self.weights(q, seen, sm_scale)
        o = w @ self.v
        w2 = w ** 2
        var = (UBF * o) ** 2 + w2 @ self.verr2 + 2.0 ** -50 * (vis.double() @ self.v ** 2) / total ** 2

        def by_score(e2):  # sum_t w_t^2 e_t^2 (v_t - o)^2
            a = w2 * e2
            return a @ self.v ** 2 - 2 * o * (a @ self.v) + o ** 2 * a.sum(1, keepdim=True)

        size = abs(sm_scale) * (q.abs() @ self.size.T)
        fp32 = 2.0 ** -20 * size + 2.0 ** -21 * abs(sm_scale) * (q @ self.kc.T).abs()
        fp32 = fp32 + 2.0 ** -22 * (torch.where(vis, s, 0.0).abs() + 1.0)
        var = var + by_score(fp32 ** 2 + sm_scale ** 2 * (q ** 2 @ (self.kerr ** 2).T))
        # the query's rounding, and per-channel centres block by block
        wk = w[:, :, None] * self.k
        move = wk.transpose(1, 2) @ self.v - wk.sum(1)[:, :, None] * o[:, None, :]  # [n][channel of q][channel of o]
        qerr = U16 * q.abs()
        if self.narrow:
            qerr = 2.0 ** -16 * (q * self.lam).abs().amax(1, keepdim=True) / self.lam
        var = var + sm_scale ** 2 * torch.einsum("nc,nco->no", qerr ** 2, move ** 2)
        for i in range(self.blocks):
            t = slice(128 * i, 128 * i + 128)
            m = w[:, t] @ self.v[t] - w[:, t].sum(1, keepdim=True) * o
            var = var + sm_scale ** 2 * (q ** 2 @ self.kblock[128 * i] ** 2)[:, None] * m ** 2
        if self.narrow:
            var = var + (2.0 ** -12 * (w @ self.vr)) ** 2
        return o, var

    def without(self, q, seen, sm_scale, tokens, times=0.0):
        """The output with the given tokens' weights multiplied by `times` (0: lost, 2: counted twice)."""
        w = self.weights(q, seen, sm_scale)[0].clone()
        w[:, tokens] *= times
        total = w.sum(1, keepdim=True)
        return torch.where(total > 0, w / total, 0.0) @ self.v


def rms(x):
    return float(x.double().pow(2).mean().sqrt())


def over(err, var):
    """By how much an error exceeds the limits above (at most 1: within them)."""
    whole = rms(err) / (1.25 * float(var.mean().sqrt()) + 1e-30)
    rows = err.pow(2).mean(-1).sqrt() / (2.5 * var.mean(-1).sqrt() + 1e-30)
    return max(whole, float(rows.max()))


def check_rms(q, dk, dv, mask, ks, vs, got, mode, bits, lam=None, sm_scale=128 ** -0.5, plant=(), streams=None, cancel=False):
    """Check an output [B][n][Hq][128]; -> the relative root mean square error of the streams looked at.

    plant: pairs (tokens, times): an output that lost those tokens of each stream (cached ones first; times 0) or counted them
    times over has to exceed the limits, three times over in the stream's root mean square."""
    B, n, Hq, _ = q.shape
    H = dk.shape[2]
    G = Hq // H
    seen = sees(mask, B, n).to(q.device)
    errs, outs = [], []
    for b, j in streams or [(b, j) for b in range(B) for j in range(H)]:
        part = lambda x: _rows(x, b, j)  # noqa: E731
        st = Stream(part(ks), part(vs), dk[b, :, j], dv[b, :, j], mode, bits, None if lam is None else lam[j], n * G <= 8 and ks.shape[2] > 0,
                    cancel)
        qs = [q[b, :, j * G + g].double() for g in range(G)]
        o, var = (torch.stack(x, 1) for x in zip(*(st.expect(x, seen[b], sm_scale) for x in qs)))
        err = got[b, :, j * G:(j + 1) * G].double() - o
        assert torch.isfinite(err).all(), (b, j)
        assert over(err, var) <= 1.0, (b, j, over(err, var), rms(err) / rms(o))
        for tokens, times in plant:
            bad = torch.stack([st.without(x, seen[b], sm_scale, tokens, times) for x in qs], 1)
            assert rms(bad - o) > 3 * 1.25 * float(var.mean().sqrt()), (b, j, tokens, times)
        errs.append(err)
        outs.append(o)
    return rms(torch.stack(errs)) / max(rms(torch.stack(outs)), 1e-30)


def _rows(x, b, j):
    y = x[b, j]
    for name in ("centre", "range"):
        if hasattr(x, name):
            setattr(y, name, getattr(x, name)[b, j])
    return y
