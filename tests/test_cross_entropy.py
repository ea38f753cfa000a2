"""lmhead_cross_entropy_f32 and lmhead_cross_entropy_grad against the formulas in 64 bits
(tests/training_reference.py, which derives the tolerances), at the sizes and masks where tiles,
pieces of the vocabulary, splits and ragged ends meet."""
import math

import pytest
import torch

import fp32_accumulate_lm_b200 as lm
from gpu_helpers import check_status
from training_reference import IGNORE, CrossEntropy, assert_close

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def make(rows, H, V, dtype="bf16", bias=False, masked=0.0, seed=0, alpha=1.0, reduction="mean",
         garbage=True):
    g = torch.Generator(device="cuda").manual_seed(1000 * rows + 10 * H + V + seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    dt = DTYPES[dtype]
    W = (normal(V, H) * (0.8 / (math.sqrt(H) * alpha))).to(dt)
    targets = torch.randint(0, V, (rows,), generator=g, device="cuda", dtype=torch.int32)
    hidden = (normal(rows, H) + W[targets.long()].float() * 4 / alpha).to(dt)
    if masked:
        out = torch.rand((rows,), generator=g, device="cuda") < masked
        targets[out] = IGNORE
        if garbage:  # what padding may hold
            hidden[out, ::2] = float("nan")
            hidden[out, 1::2] = float("inf")
    b = (normal(V) * 0.5).to(dt) if bias else None
    gl = normal(rows) / rows if reduction == "none" else torch.tensor(0.75, device="cuda")
    return hidden, W, targets, b, gl


def run_both(hidden, W, targets, b, gl, **how):
    loss, lse = lm.cross_entropy_f32(hidden, W, targets, bias=b, **how)
    grads = lm.cross_entropy_grad(hidden, W, targets, lse, gl, bias=b, **how)
    check_status()
    ref = CrossEntropy(hidden, W, targets, bias=b, grad_loss=gl, **how)
    return loss, lse, grads, ref


def compare(loss, lse, grads, ref):
    assert_close(lse, ref.lse, ref.lse_tol, "lse")
    assert_close(loss, ref.loss, ref.loss_tol, "loss")
    assert_close(grads[0], ref.d_hidden, ref.d_hidden_tol, "d_hidden")
    assert_close(grads[1], ref.d_W, ref.d_W_tol, "d_W")
    if grads[2] is not None:
        assert_close(grads[2], ref.d_bias, ref.d_bias_tol, "d_bias")


# rows around the lone-CTA and pair tiles, vocabularies around the 128- and 256-wide ones, hidden
# sizes that end inside a K step and a tile
SIZES = [(1, 8, 1), (1, 64, 127), (3, 8, 5), (4, 256, 1024), (31, 72, 129), (127, 200, 255),
         (128, 64, 300), (129, 64, 300), (130, 136, 257), (255, 264, 256), (256, 64, 512),
         (257, 520, 513), (300, 512, 4097), (1000, 128, 8200)]


@pytest.mark.parametrize("rows,H,V", SIZES)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_sizes(rows, H, V, dtype):
    args = make(rows, H, V, dtype)
    compare(*run_both(*args, ignore_index=None))


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("rows,H,V,masked", [(7, 64, 300, 0.5), (128, 136, 700, 0.3),
                                             (400, 72, 1000, 0.4), (513, 256, 600, 0.9)])
def test_masked_rows_bias_alpha_and_z_loss(rows, H, V, masked, dtype, reduction):
    args = make(rows, H, V, dtype, bias=True, masked=masked, alpha=0.25, reduction=reduction)
    compare(*run_both(*args, alpha=0.25, z_loss=1e-3, reduction=reduction))
