"""The precision of the training gradients where the elementwise bounds of tests/training_reference.py
are too wide to tell: d_bias summed in fp32. The tests on the CPU show that the bounds tell the
kernels' roundings from wrong ones."""
import math

import pytest
import torch

import fp32_accumulate_lm_b200 as lm
from gpu_helpers import check_status
from training_precision import IGNORE, Centred, rounded
from training_reference import assert_close, half_step

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def make(device, rows, H, V, dtype="bf16", reduction="none", masked=0.0, targets="any", seed=0,
         sure=0.0):
    """targets: "any", or "twice": every target again half the rows later. sure: how many units of
    logit the row has for an entry that is not its target."""
    g = torch.Generator(device=device).manual_seed(100 * rows + V + seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device=device)

    dt = DTYPES[dtype]
    W = (normal(V, H) * (0.8 / math.sqrt(H))).to(dt)
    if targets == "twice":
        half = (rows + 1) // 2
        assert V >= half
        t = torch.randperm(V, generator=g, device=device)[:half].repeat(2)[:rows]
    else:
        t = torch.randint(0, V, (rows,), generator=g, device=device)
    hidden = normal(rows, H)
    if sure:
        wrong = W[(t + 1) % V].float()
        hidden = 0.1 * hidden + wrong * (sure / wrong.square().sum(1, keepdim=True))
    t = t.to(torch.int32)
    if masked:
        out = torch.rand((rows,), generator=g, device=device) < masked
        t[out] = IGNORE
        hidden[out] = float("nan")
    gl = normal(rows) / rows if reduction == "none" else torch.tensor(0.75, device=device)
    bias = (normal(V) * 0.5).to(dt)
    return hidden.to(dt), W, t, bias, gl


# ------------------------------------------------------------------ d_bias

def bias_bound(c, base=None):
    """Elementwise, for a sum of d in fp32 that is rounded once: each entry of d off by its logit's
    error and its exponential's (2^-20), the sum by n 2^-23 of the sizes."""
    size = c.d.abs().sum(0) * abs(c.alpha * c.scale)
    want = c.d_bias(c.d) + (0.0 if base is None else base.double())
    u = half_step(c.dtype)
    tol = size * (c.logits + 2.0 ** -20 + min(1e-4, c.t.numel() * 2.0 ** -23)) + u * want.abs()
    if base is not None:
        tol = tol + 2.0 ** -23 * base.double().abs()
    return want, tol + torch.finfo(c.dtype).smallest_normal * u


@pytest.mark.parametrize("rows,dtype", [(3, "bf16"), (40, "bf16"), (300, "bf16"), (3, "f16"),
                                        (20, "f16")])
def test_the_bound_of_d_bias_tells_sums_of_rounded_entries(rows, dtype):
    hidden, W, t, b, gl = make("cpu", rows, 64, 3000, dtype)
    c = Centred(hidden, W, t, bias=b, reduction="none", grad_loss=gl)
    want, tol = bias_bound(c)
    assert_close(rounded(c.d_bias(c.d), c.dtype), want, tol, "d_bias")
    with pytest.raises(AssertionError):
        assert_close(rounded(c.d_bias(c.round_d()), c.dtype), want, tol, "d_bias")


def gradients(hidden, W, t, b, gl, reduction, **kw):
    loss, lse = lm.cross_entropy_f32(hidden, W, t, bias=b, reduction=reduction)
    got = lm.cross_entropy_grad(hidden, W, t, lse, gl, bias=b, reduction=reduction, **kw)
    check_status()
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("rows,V,masked", [(3, 3000, 0.0), (40, 3000, 0.0), (300, 3000, 0.3),
                                           (1000, 70, 0.0), (2100, 130001, 0.1)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_d_bias_is_summed_in_fp32(rows, V, masked, dtype):
    """Lone CTAs, pairs and big tiles, masked rows, added to what is there, and alone."""
    hidden, W, t, b, gl = make("cuda", rows, 64, V, dtype, masked=masked)
    c = Centred(hidden, W, t, bias=b, reduction="none", grad_loss=gl)
    want, tol = bias_bound(c)
    got = gradients(hidden, W, t, b, gl, "none")[2]
    assert_close(got, want, tol, "d_bias")
    alone = torch.empty_like(b)
    gradients(hidden, W, t, b, gl, "none", out=(None, None, alone))
    assert torch.equal(alone, got)
    base = (b.float() / rows).to(b.dtype)
    added = base.clone()
    gradients(hidden, W, t, b, gl, "none", out=(None, None, added), accumulate=True)
    assert_close(added, *bias_bound(c, base), "d_bias, added")
