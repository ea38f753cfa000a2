"""The training operators by their definitions, in 64 bits, and how far the kernels may be off.

Cross entropy. With u = half a step of the operands' 16-bit type (finfo.eps / 2), and for each row
    dz_r = max_v min(1e-4, H 2^-23) * alpha * sum_k |h_k w_vk| + alpha-rounding
the largest error of a logit of the row (an fp32 sum of H exact products in an unknown order errs by
less than H 2^-24 of the sum of their sizes; 1e-4 is the bound the head's own tests use):
  * lse_r, and z at the target, are each off by at most dz_r plus the fp32 reduction: the running
    sum passes ceil(V / 128) / 32 + 40 merges, each two roundings and an exponential (2^-21 each,
    counted generously), and the final log and additions round once each (2^-22 of the values);
  * an entry of d is off by the relative error of its exponential, 2 dz_r + 2^-20, before it is
    rounded to 16 bits, u relative, so d_hidden and d_W are off by at most
    scale * (u + 2 dz_r + 2^-20) * (|d| @ |W|) (or (|d|^T @ |h|)), where |d| counts the softmax term
    and the target's 1 apart, plus the fp32 sums (1e-4 of the same, as above, at most (K) 2^-23),
    plus the final rounding, u of the value, and half the smallest subnormal;
  * a softmax value below 2^-126 may be 0 (fp32's normal range): 2^-126 of the factor;
  * with fp16 an entry below 2^-14 of the scaled range is off by half a subnormal step instead:
    2^-25 of a range whose largest factor is at least 2^13: 2^-38 of that factor.
"""
import torch

IGNORE = -100


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def sum_bound(n):
    """Relative error of an fp32 sum of n products, as a share of the sum of their sizes."""
    return min(1e-4, n * 2.0 ** -23) + 2.0 ** -23


class CrossEntropy:
    """Loss, lse and gradients of one call in 64 bits, each with its bound (`*_tol`)."""

    def __init__(self, hidden, W, targets, alpha=1.0, bias=None, ignore_index=IGNORE, z_loss=0.0,
                 reduction="mean", grad_loss=None, base_W=None, base_bias=None):
        R, H = hidden.shape
        V = W.shape[0]
        dtype, u, dev = hidden.dtype, half_step(hidden.dtype), hidden.device
        counts = torch.ones(R, dtype=torch.bool, device=dev) if ignore_index is None else \
            targets != ignore_index
        rows = counts.nonzero()[:, 0]
        n = rows.numel()
        h, w, t = hidden[rows].double(), W.double(), targets[rows].long()
        bad = (t < 0) | (t >= V)
        t = t.clamp(0, V - 1)
        z = h @ w.t()
        size = h.abs() @ w.abs().t()
        if bias is not None:
            z = z + bias.double()
            finite = torch.where(torch.isfinite(bias.double()), bias.double().abs(), 0.0)
            size = size + finite
        z = z * alpha
        dz = (size * abs(alpha)).amax(1) * sum_bound(H) if n else torch.zeros(0, device=dev)
        lse = torch.logsumexp(z, 1) if n else z.new_zeros(0)
        zt = z.gather(1, t[:, None])[:, 0]
        each = lse - zt + z_loss * lse ** 2
        each = torch.where(bad, float("nan"), each)
        merges = (V + 127) // 128 / 32 + 40
        lse_tol = dz + merges * 2.0 ** -21 + 2.0 ** -22 * (1 + lse.abs())
        each_tol = (lse_tol + dz) * (1 + 2 * z_loss * lse.abs()) + \
            2.0 ** -21 * (1 + lse.abs() + zt.abs() + z_loss * lse ** 2)

        def spread(x, fill=0.0):
            whole = torch.full((R, *x.shape[1:]), fill, dtype=torch.float64, device=dev)
            whole[rows] = x.double()
            return whole

        self.lse, self.lse_tol = spread(lse), spread(lse_tol)
        if reduction == "none":
            self.loss, self.loss_tol = spread(each), spread(each_tol)
        else:
            d = max(n, 1) if reduction == "mean" else 1
            self.loss = each.sum() / d
            self.loss_tol = (each_tol.sum() + each.abs().sum() * (R / 1024 + 12) * 2.0 ** -24) / d \
                + 2.0 ** -22 * self.loss.abs()
        if grad_loss is None:
            return
        g = grad_loss.double()
        g = g[rows] if reduction == "none" else \
            (g.reshape(()) / (max(n, 1) if reduction == "mean" else 1)).expand(n)
        g = torch.where(bad, float("nan"), g)
        a = (g * (1 + 2 * z_loss * lse))[:, None]
        p = torch.exp(z - lse[:, None])
        d = a * p
        d[torch.arange(n, device=dev), t] -= g
        off = (p * a.abs()) * (u + 2 * dz[:, None] + 2.0 ** -20) + a.abs() * 2.0 ** -126
        off[torch.arange(n, device=dev), t] += g.abs() * (u + 2.0 ** -22)
        if dtype == torch.float16 and n:
            top = torch.maximum(a.abs().max(), g.abs().max()) if reduction == "none" else a.abs().max()
            off = off + top * 2.0 ** -38
        d, off = d * alpha, off * abs(alpha)
        tiny = torch.finfo(dtype).smallest_normal * u

        def done(value, tol):
            return value, tol + u * value.abs() + tiny

        size = d.abs() + off
        self.d_hidden, self.d_hidden_tol = done(
            spread(d @ w), spread(off @ w.abs() + sum_bound(V) * (size @ w.abs())))
        base = 0.0 if base_W is None else base_W.double()
        self.d_W, self.d_W_tol = done(
            base + d.t() @ h, off.t() @ h.abs() + sum_bound(max(n, 1)) * (size.t() @ h.abs())
            + 2.0 ** -23 * (torch.zeros((), device=dev) if base_W is None else base.abs()))
        base = 0.0 if base_bias is None else base_bias.double()
        self.d_bias, self.d_bias_tol = done(
            base + d.sum(0), off.sum(0) + sum_bound(max(n, 1)) * size.sum(0)
            + 2.0 ** -23 * (torch.zeros((), device=dev) if base_bias is None else base.abs()))


def assert_close(got, want, tol, what):
    got = got.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), \
        f"{what}: {int((torch.isnan(got) != nan).sum())} values are NaN on one side only"
    off = torch.where(nan, 0.0, (got - want).abs())
    tol = torch.where(nan, 0.0, tol)
    bad = ~(off <= tol)
    if bad.any():
        worst = int((off / tol.clamp(min=1e-300)).reshape(-1).argmax())
        at = torch.unravel_index(torch.tensor(worst), got.shape) if got.dim() else ()
        raise AssertionError(
            f"{what}: {int(bad.sum())} of {bad.numel()} outside the bound; worst at "
            f"{tuple(int(i) for i in at)}: {float(got.reshape(-1)[worst])!r} for "
            f"{float(want.reshape(-1)[worst])!r}, bound {float(tol.reshape(-1)[worst])!r}")


def embedding(ids, W, scale=1.0, v_begin=0):
    """(rows, bound): one fp32 multiply and one rounding."""
    local = ids.long() - v_begin
    held = (local >= 0) & (local < W.shape[0])
    rows = W.double()[local.clamp(0, W.shape[0] - 1)] * scale
    rows = torch.where(held[..., None], rows, 0.0)
    u = half_step(W.dtype)
    return rows, (u + 2.0 ** -23) * rows.abs() + torch.finfo(W.dtype).smallest_normal * u


def embedding_grad(d_out, ids, V, scale=1.0, v_begin=0, base=None):
    """(d_W, bound): an fp32 sum of n terms in any order errs by less than n 2^-24 of the sum of
    their sizes; then the scale, the base's addition and the rounding to 16 bits."""
    H = d_out.shape[-1]
    flat, local = d_out.reshape(-1, H), ids.reshape(-1).long() - v_begin
    at = ((local >= 0) & (local < V)).nonzero()[:, 0]
    rows, local = flat[at].double(), local[at]
    d_W = torch.zeros((V, H), dtype=torch.float64, device=d_out.device)
    size = torch.zeros_like(d_W)
    d_W.index_add_(0, local, rows)
    size.index_add_(0, local, rows.abs())
    n = torch.bincount(local, minlength=V).double()[:, None]
    tol = abs(scale) * size * (n + 2) * 2.0 ** -24
    d_W = d_W * scale
    if base is not None:
        d_W = d_W + base.double()
        tol = tol + 2.0 ** -23 * base.double().abs()
    u = half_step(d_out.dtype)
    return d_W, tol + (u + 2.0 ** -23) * d_W.abs() + torch.finfo(d_out.dtype).smallest_normal * u
