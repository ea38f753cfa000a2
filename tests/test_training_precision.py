"""The precision of the training gradients where the elementwise bounds of tests/training_reference.py
are too wide to tell: the target's entry of d put back in fp32 (tests/training_precision.py derives
the bounds), d_bias summed in fp32. The tests on the CPU show that the bounds tell the kernels'
roundings from wrong ones."""
import math

import pytest
import torch

import fp32_accumulate_lm_b200 as lm
from gpu_helpers import check_status
from training_precision import IGNORE, Centred, assert_as_foretold, rounded
from training_reference import CrossEntropy, assert_close, half_step

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


def gradients(hidden, W, t, b, gl, reduction, **kw):
    loss, lse = lm.cross_entropy_f32(hidden, W, t, bias=b, reduction=reduction)
    got = lm.cross_entropy_grad(hidden, W, t, lse, gl, bias=b, reduction=reduction, **kw)
    check_status()
    return got


# ------------------------------------------------------------------ the target's entry of d

CPU_SIZES = [(96, 64, 1500, "bf16", "none", "any"), (300, 64, 700, "f16", "none", "any"),
             (1000, 64, 600, "bf16", "none", "twice"), (500, 64, 900, "bf16", "mean", "any")]


@pytest.mark.parametrize("rows,H,V,dtype,reduction,targets", CPU_SIZES)
def test_the_bounds_tell_a_missing_mend(rows, H, V, dtype, reduction, targets):
    hidden, W, t, b, gl = make("cpu", rows, H, V, dtype, reduction, targets=targets)
    c = Centred(hidden, W, t, bias=b, reduction=reduction, grad_loss=gl)
    dt = DTYPES[dtype]

    def outputs(mend):
        got = c.outputs(c.round_d(mend))
        return [rounded(x, dt) for x in got[:2]] + [rounded(c.d_bias(c.d), dt)]

    assert_as_foretold(c, outputs("target"))
    # a d that is off by what its logits may be rounds some entries the other way
    c.d *= 1 + c.logits * (2 * torch.rand(c.d.shape, generator=torch.Generator().manual_seed(1)) - 1)
    moved = outputs("target")
    c = Centred(hidden, W, t, bias=b, reduction=reduction, grad_loss=gl)
    assert_as_foretold(c, moved)
    for wrong in ("nothing", "flipped") + (("first",) if targets == "twice" else ()):
        for i in (0, 1):
            if wrong == "first" and i == 0:
                continue
            got = [None] * 3
            got[i] = outputs(wrong)[i]
            with pytest.raises(AssertionError):
                assert_as_foretold(c, got)


CASES = [
    (96, 64, 2000, "bf16", "none", 0.0, "any"),         # lone CTAs
    (300, 64, 3000, "f16", "none", 0.3, "any"),         # pairs, masked rows
    (700, 72, 9000, "bf16", "mean", 0.0, "any"),
    (12000, 64, 7000, "bf16", "none", 0.0, "twice"),    # targets again 6000 rows later
    (12001, 64, 7000, "f16", "none", 0.1, "twice"),
    (16640, 64, 10001, "bf16", "none", 0.2, "any"),     # pieces of the vocabulary
    (2100, 72, 130001, "bf16", "none", 0.0, "any"),     # big tiles
]


@pytest.mark.gpu
@pytest.mark.parametrize("rows,H,V,dtype,reduction,masked,targets", CASES)
def test_gradients_are_as_far_off_as_foretold(rows, H, V, dtype, reduction, masked, targets):
    """Written, and added to buffers that hold values of the gradient's own size."""
    hidden, W, t, b, gl = make("cuda", rows, H, V, dtype, reduction, masked, targets)
    c = Centred(hidden, W, t, bias=b, reduction=reduction, grad_loss=gl)
    assert_as_foretold(c, gradients(hidden, W, t, b, gl, reduction))
    g = torch.Generator(device="cuda").manual_seed(9)
    base_W, base_b = ((torch.randn(x.shape, generator=g, device="cuda") * x.square().mean().sqrt())
                      .to(hidden.dtype) for x in (c.d_W(c.d), c.d_bias(c.d)))
    out = (None, base_W.clone(), base_b.clone())
    gradients(hidden, W, t, b, gl, reduction, out=out, accumulate=True)
    assert_as_foretold(c, out, base_W, base_b)


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


# ------------------------------------------------------------------ weights

def step(hidden, W, t, gl, alpha=1.0):
    loss, lse = lm.cross_entropy_f32(hidden, W, t, alpha=alpha, reduction="none")
    grads = lm.cross_entropy_grad(hidden, W, t, lse, gl, alpha=alpha, reduction="none")
    check_status()
    return grads, CrossEntropy(hidden, W, t, alpha=alpha, reduction="none", grad_loss=gl)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [40, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("log2", [(120, -110), (126, -116), (-100, 90)])
def test_weights_as_far_from_1_as_alpha(rows, dtype, log2):
    """Upstream gradients near fp32's limits, which alpha brings back: fp16's range holds the entries
    of d without either."""
    hidden, W, t, _, gl = make("cuda", rows, 64, 500, dtype)
    up, alpha = 2.0 ** log2[0], 2.0 ** log2[1]
    if alpha > 1:  # all logits 0: what alpha would make of them fp32 could not hold
        W.zero_()
    grads, ref = step(hidden, W, t, gl.clamp(-1.9, 1.9) * up, alpha)
    assert_close(grads[0], ref.d_hidden, ref.d_hidden_tol, "d_hidden")
    assert_close(grads[1], ref.d_W, ref.d_W_tol, "d_W")


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [60, 300])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_weights_of_very_different_sizes(rows, dtype):
    """Down to 2^-28 of the largest. The power of two is common to the call: an entry of fp16's d is
    off by half a step, or by 2^-38 of the largest factor where that is more."""
    hidden, W, t, _, gl = make("cuda", rows, 64, 3000, dtype)
    gl = gl.sign() * 2.0 ** -(torch.arange(rows, device="cuda") % 29).float() * 4096
    grads, ref = step(hidden, W, t, gl)
    assert_close(grads[0], ref.d_hidden, ref.d_hidden_tol, "d_hidden")
    assert_close(grads[1], ref.d_W, ref.d_W_tol, "d_W")


# ------------------------------------------------------------------ rows sure of a wrong entry

@pytest.mark.gpu
@pytest.mark.parametrize("rows,V", [(96, 3000), (700, 3000), (2100, 130001)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_rows_sure_of_a_wrong_entry(rows, V, dtype):
    """Their entry of d at the wrong entry is as large as the target's and is rounded to 16 bits
    unmended: the errors are those foretold, past what rounding the gradients alone gives."""
    hidden, W, t, b, gl = make("cuda", rows, 64, V, dtype, sure=math.log(V) + 1)
    c = Centred(hidden, W, t, reduction="none", grad_loss=gl)
    p = (c.d / gl.double()[c.rows][:, None])[c.at, (c.t + 1) % V]
    assert 0.3 < float(p.mean()) < 0.95
    loss, lse = lm.cross_entropy_f32(hidden, W, t, reduction="none")
    got = lm.cross_entropy_grad(hidden, W, t, lse, gl, reduction="none")
    check_status()
    assert_as_foretold(c, got)


# ------------------------------------------------------------------ the loss of rows sure of their target

@pytest.mark.gpu
@pytest.mark.parametrize("rows,V", [(1, 1024), (40, 1024), (300, 5000)])
def test_small_losses_keep_their_bits(rows, V):
    """Logits that fp32 holds exactly in any order of summation (multiples of 2^-8 below 2^8), so all
    that is off comes behind them. Each term of the sum, 2^(x - x_t) with x = z log2(e), is off by the
    rounding of log2(e), of x and of x_t, |x| 2^-24 each, in the exponent (times log 2), by 2^-22 in
    exp2 and by its way through at most 60 sums and rescalings, 2^-22 each, and log1p by 2^-22."""
    g = torch.Generator(device="cuda").manual_seed(rows + V)
    H = 64
    W = torch.randint(-4, 5, (V, H), generator=g, device="cuda").float() / 16
    t = torch.randint(0, V, (rows,), generator=g, device="cuda")
    hidden = torch.randint(-8, 9, (rows, H), generator=g, device="cuda").float() / 16
    # units along the target's row, for a loss of 1e-1 to 1e-5
    lead = torch.randint(2, 5, (rows, 1), generator=g, device="cuda").float()
    hidden += W[t].sign() * lead
    hidden, W, t = hidden.bfloat16(), W.bfloat16(), t.to(torch.int32)
    z = hidden.double() @ W.double().t()
    assert float(z.abs().max()) < 2 ** 8 and torch.equal(z * 2 ** 8, (z * 2 ** 8).round())
    zt = z.gather(1, t.long()[:, None])
    others = z.scatter(1, t.long()[:, None], float("-inf"))
    want = torch.log1p(torch.exp(others - zt).sum(1))
    loss, lse = lm.cross_entropy_f32(hidden, W, t, reduction="none")
    check_status()
    assert float(want.min()) < 1e-4 or rows == 1
    x = z.abs().amax(1) * 1.4427
    tol = want * ((4 * x) * 2.0 ** -24 * 0.6932 + 63 * 2.0 ** -22)
    assert_close(loss, want, tol, "loss")
