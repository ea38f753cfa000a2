"""lmhead_embedding and lmhead_embedding_grad against the formulas in 64 bits, at the sizes and id
patterns where the sort's tiles and digits, the sums' tiles and runs across them meet."""
import pytest
import torch

import fp32_accumulate_lm_b200 as lm
import training_reference as ref
from gpu_helpers import check_status
from training_reference import assert_close

pytestmark = pytest.mark.gpu

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def normal(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def draw_ids(pattern, tokens, V, seed=0):
    g = torch.Generator(device="cuda").manual_seed(7 * tokens + V + seed)

    def rand(high, n=tokens):
        return torch.randint(0, high, (n,), generator=g, device="cuda", dtype=torch.int32)

    ids = rand(V)
    if pattern == "one":        # a single run through every tile
        ids = torch.full_like(ids, V // 2)
    elif pattern == "half":     # one heavy id among others
        ids[rand(2) == 0] = V - 1
    elif pattern == "few":      # runs a few tiles long
        ids = rand(min(V, 5))
    elif pattern == "absent":   # ids outside the table on both sides
        lot = rand(4)
        ids[lot == 0] = -1
        ids[lot == 1] = V
        ids[rand(50) == 0] = 2 ** 31 - 1
        ids[rand(50) == 0] = -2 ** 31
    elif pattern == "none":
        ids = torch.full_like(ids, -1)
    elif pattern == "sorted":
        ids = torch.sort(ids).values
    return ids


@pytest.mark.parametrize("tokens,H,V", [(1, 8, 1), (1, 2048, 1000), (7, 72, 10), (65, 1032, 333),
                                        (300, 264, 5000)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_embedding(tokens, H, V, dtype):
    W = normal(V, V, H, dtype=DTYPES[dtype])
    for pattern, scale in (("spread", 1.0), ("absent", 45.25), ("one", 0.3)):
        ids = draw_ids(pattern, tokens, V)
        out = lm.embedding(ids, W, scale=scale)
        check_status()
        want, tol = ref.embedding(ids, W, scale)
        assert_close(out, want, tol, f"{pattern}")
        if scale == 1.0:
            assert torch.equal(out, W[ids.long()])


@pytest.mark.parametrize("pattern", ["spread", "one", "half", "few", "absent", "none", "sorted"])
@pytest.mark.parametrize("tokens,H,V", [(1, 8, 1), (2, 64, 3), (63, 72, 100), (64, 264, 511),
                                        (65, 520, 512), (129, 1032, 513), (1000, 64, 40),
                                        (1025, 136, 5003), (9000, 72, 300), (17000, 64, 262144)])
def test_grad(tokens, H, V, pattern):
    dtype = DTYPES["f16" if tokens % 2 else "bf16"]
    ids = draw_ids(pattern, tokens, V)
    d_out = normal(tokens + H, tokens, H, dtype=dtype)
    d_out[(ids < 0) | (ids >= V)] = float("nan")  # reaches nothing
    d_W = lm.embedding_grad(d_out, ids, V, scale=1.5)
    check_status()
    want, tol = ref.embedding_grad(d_out, ids, V, 1.5)
    assert_close(d_W, want, tol, pattern)
    # added to what is there: rows without a token stay as they are, bit for bit
    base = normal(V, V, H, dtype=dtype)
    out = base.clone()
    lm.embedding_grad(d_out, ids, V, scale=1.5, accumulate=True, out=out)
    check_status()
    want, tol = ref.embedding_grad(d_out, ids, V, 1.5, base=base)
    assert_close(out, want, tol, f"{pattern}, accumulated")
    seen = torch.zeros(V, dtype=torch.bool, device="cuda")
    seen[ids[(ids >= 0) & (ids < V)].long()] = True
    assert torch.equal(out[~seen], base[~seen])
