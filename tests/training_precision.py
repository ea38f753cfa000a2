"""How far off the cross entropy's gradients are in the 2-norm, foretold from the roundings that the
kernels make (test infrastructure; computed in 64 bits on any device).

d is rounded to the operands' 16-bit type before the products of d_hidden and d_W, but for the
target's entry, which enters them exactly (what its rounding loses is put back in fp32). d_bias is
summed from d in fp32. Then each output is rounded once. So
    error = |round16(G(round_d(d))) - G(d)|,       G the gradient as a function of d,
for which `foretold` takes the rounding of the very d of the call, the power of two taken out as the
kernels take it out for fp16. What is not foretold: a logit is an fp32 sum of H products in an
unknown order, off by at most 2 H 2^-24 sum |h_k w_vk| (its truncations counted as twice a rounding),
and with it the whole entry of d, relatively, so that some entries round the other way; it joins as
the root of the sum of squares, since those moves do not follow the roundings' signs. The sums over
rows and vocabulary and their fp32 roundings are smaller by 2^-12. SLACK covers the spread of a norm
over a few thousand roundings (1 / sqrt(2 n), 2 % for n = 1500).
"""
import torch

SLACK = 1.03
IGNORE = -100


class Centred:
    """d of a call in 64 bits, without alpha: rows that count, their targets, their hidden rows."""

    def __init__(self, hidden, W, targets, alpha=1.0, bias=None, ignore_index=IGNORE, z_loss=0.0,
                 reduction="mean", grad_loss=None):
        counts = torch.ones_like(targets, dtype=torch.bool) if ignore_index is None else \
            targets != ignore_index
        self.rows = counts.nonzero()[:, 0]
        self.total, self.dtype, self.alpha = hidden.shape[0], hidden.dtype, alpha
        n = self.rows.numel()
        self.at = torch.arange(n, device=hidden.device)
        self.h, self.w, self.t = hidden[self.rows].double(), W.double(), targets[self.rows].long()
        z = self.h @ self.w.t()
        if bias is not None:
            z += bias.double()
        z *= alpha
        lse = torch.logsumexp(z, 1)
        self.lse = lse
        if reduction == "none":
            g, self.scale = grad_loss.double()[self.rows], 1.0
        else:
            g = torch.ones_like(lse)
            self.scale = float(grad_loss) / (max(n, 1) if reduction == "mean" else 1)
        a = g * (1 + 2 * z_loss * lse)
        self.d = torch.exp_(z.sub_(lse[:, None])).mul_(a[:, None])
        self.d[self.at, self.t] -= g
        top = float(torch.maximum(a.abs().max(), g.abs().max())) if n else 1.0
        self.up = 2.0 ** (13 - int(torch.tensor(top, dtype=torch.float64).log2().floor()))
        # the relative error of an entry of d that its logit's fp32 sum may bring
        size = max((float((h.abs() @ self.w.abs().t()).max()) for h in self.h.split(256)), default=0.0)
        self.logits = abs(alpha) * size * 2 * hidden.shape[1] * 2.0 ** -24

    def round_d(self, mend="target"):
        """d as the products have it. Wrong forms for the tests of these bounds: "nothing" mends no
        entry, "flipped" takes the lost part away once more, "first" mends the first row of each
        target only."""
        x = self.d * self.up
        r = x.float().to(self.dtype).double()
        at, t = self.at, self.t
        exact, rounded = x[at, t], r[at, t]
        if mend == "target":
            r[at, t] = exact
        elif mend == "flipped":
            r[at, t] = 2 * rounded - exact
        elif mend == "first":
            first = torch.full((self.w.shape[0],), at.numel(), device=t.device, dtype=torch.long)
            first.scatter_reduce_(0, t, at, "amin")
            mine = first[t] == at
            r[at[mine], t[mine]] = exact[mine]
        return r.div_(self.up)

    def d_hidden(self, d):
        whole = torch.zeros((self.total, self.w.shape[1]), dtype=torch.float64, device=d.device)
        whole[self.rows] = (d @ self.w) * (self.alpha * self.scale)
        return whole

    def d_W(self, d):
        return (d.t() @ self.h) * (self.alpha * self.scale)

    def d_bias(self, d):
        return d.sum(0) * (self.alpha * self.scale)

    def outputs(self, d, base_W=None, base_bias=None):
        """(d_hidden, d_W, d_bias) for this d, in 64 bits."""
        w, b = self.d_W(d), self.d_bias(d)
        return (self.d_hidden(d), w if base_W is None else w + base_W.double(),
                b if base_bias is None else b + base_bias.double())


def rounded(x, dtype):
    return x.float().to(dtype).double()


def error(got, want):
    return float((got.double() - want).norm())


def foretold(c, exact, as_used, own):
    """The largest 2-norm of an output's error: `exact` it is, `as_used` it would be with d as the
    products have it, `own` the size of the part that the logits' errors act on."""
    e = error(rounded(as_used, c.dtype), exact)
    return SLACK * (e ** 2 + (c.logits * float(own.norm())) ** 2) ** 0.5


def assert_as_foretold(c, got, base_W=None, base_bias=None):
    """got = (d_hidden, d_W, d_bias), any of them None: each as a whole, d_W also on the rows that are
    some row's target and on the others."""
    exact = c.outputs(c.d, base_W, base_bias)
    used = c.round_d()
    as_used = c.outputs(used, base_W, base_bias)[:2] + (exact[2],)
    own = c.outputs(c.d)
    hit = torch.zeros(c.w.shape[0], dtype=torch.bool, device=c.d.device)
    hit[c.t] = True
    for i, name in enumerate(("d_hidden", "d_W", "d_bias")):
        if got[i] is None:
            continue
        parts = [("", slice(None))]
        if i == 1:
            parts += [(" of the targets", hit), (" of the other entries", ~hit)]
        for what, at in parts:
            off = error(got[i][at], exact[i][at])
            most = foretold(c, exact[i][at], as_used[i][at], own[i][at])
            assert off <= most, (name + what, off / most)
