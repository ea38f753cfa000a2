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


def test_many_tokens_of_one_id():
    """More entries than a turn of the sort's CTAs holds (the digits are counted first), and a run
    over all tiles."""
    tokens, H, V = 70000, 64, 1000
    for pattern in ("spread", "one", "half"):
        ids = draw_ids(pattern, tokens, V)
        d_out = normal(5, tokens, H)
        got = lm.embedding_grad(d_out, ids, V)
        check_status()
        want, tol = ref.embedding_grad(d_out, ids, V)
        assert_close(got, want, tol, pattern)


@pytest.mark.parametrize("V", [1, 511, 512, 2 ** 18 - 1, 2 ** 18, 600000])
def test_digits_of_the_sort(V):
    """Ids at both ends of each digit's range, and tables that need one, two and three passes."""
    ids = torch.tensor([0, V - 1, V // 2, V - 1, 0, V, -1, 511, 512, 513, 262143, 262144, V - 1],
                       dtype=torch.int32, device="cuda").repeat(9)
    d_out = normal(3, ids.numel(), 8)
    got = lm.embedding_grad(d_out, ids, V)
    check_status()
    want, tol = ref.embedding_grad(d_out, ids, V)
    assert_close(got, want, tol, f"V={V}")


def test_tables_larger_than_the_sort_clears():
    """Rows without a token are cleared in two launches; the boundary between them shows nowhere."""
    V, H = 70000, 1032
    for tokens in (1, 700):
        ids = draw_ids("spread", tokens, V)
        d_out = normal(tokens, tokens, H)
        out = torch.full((V, H), float("nan"), dtype=torch.bfloat16, device="cuda")
        lm.embedding_grad(d_out, ids, V, out=out)
        check_status()
        want, tol = ref.embedding_grad(d_out, ids, V)
        assert_close(out, want, tol, f"{tokens} tokens")


def test_slices_of_a_table():
    """A table split by vocabulary: the slices' embeddings add up to the whole table's, their
    gradients are its rows."""
    V, H, tokens = 1000, 72, 500
    W, d_out = normal(1, V, H), normal(2, tokens, H)
    ids = draw_ids("absent", tokens, V)
    whole, grad = lm.embedding(ids, W, scale=2.0), lm.embedding_grad(d_out, ids, V, scale=2.0)
    total = torch.zeros_like(whole)
    for rank in range(3):
        v0, n = lm.vocab_shard(V, 3, rank)
        total += lm.embedding(ids, W[v0:v0 + n].contiguous(), scale=2.0, v_begin=v0)
        part = lm.embedding_grad(d_out, ids, n, scale=2.0, v_begin=v0)
        want, tol = ref.embedding_grad(d_out, ids, n, 2.0, v0)
        assert_close(part, want, tol, f"slice {rank}")
    check_status()
    assert torch.equal(total, whole)
    # the last ids of the int32 range
    v0 = 2 ** 31 - 100
    top = torch.tensor([2 ** 31 - 1, v0, v0 - 1, -1, -2 ** 31], dtype=torch.int32, device="cuda")
    got = lm.embedding(top, W[:100].contiguous(), v_begin=v0)
    assert torch.equal(got[0], W[99]) and torch.equal(got[1], W[0])
    assert torch.count_nonzero(got[2:]) == 0


def test_shapes_and_no_tokens():
    W = normal(1, 50, 16)
    ids = draw_ids("spread", 24, 50).view(2, 3, 4)
    out = lm.embedding(ids, W)
    assert out.shape == (2, 3, 4, 16) and torch.equal(out, W[ids.long()])
    grad = lm.embedding_grad(out, ids, 50)
    want, tol = ref.embedding_grad(out, ids, 50)
    assert_close(grad, want, tol, "grad")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    empty = lm.embedding(none, W)
    assert empty.shape == (0, 16)
    assert torch.count_nonzero(lm.embedding_grad(empty, none, 50)) == 0
    base = W.clone()
    lm.embedding_grad(empty, none, 50, accumulate=True, out=base)
    assert torch.equal(base, W)
    check_status()


def test_special_values_pass_through():
    W = normal(1, 20, 8, dtype=torch.float16)
    W[3, 2], W[4, 1], W[5, 0] = float("nan"), float("inf"), 65504.0
    ids = torch.tensor([3, 4, 5, -1], dtype=torch.int32, device="cuda")
    out = lm.embedding(ids, W, scale=2.0)
    assert torch.isnan(out[0, 2]) and out[1, 1] == float("inf") and out[2, 0] == float("inf")
    assert torch.count_nonzero(out[3]) == 0
    out = lm.embedding(ids, W, scale=float("nan"))
    assert torch.isnan(out[:3]).all() and torch.count_nonzero(out[3]) == 0
    grad = lm.embedding_grad(W[:4].contiguous(), ids, 20)
    assert torch.equal(grad[3], W[0]) and torch.count_nonzero(grad[0]) == 0


def test_same_bits_every_time_other_streams_and_capture():
    tokens, H, V = 3000, 136, 700
    ids, d_out, W = draw_ids("half", tokens, V), normal(1, tokens, H), normal(2, V, H)
    first = lm.embedding_grad(d_out, ids, V)
    for _ in range(4):
        assert torch.equal(lm.embedding_grad(d_out, ids, V), first)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    a = lm.embedding_grad(d_out, ids, V, stream=s)
    c = lm.embedding(ids, W, stream=s.cuda_stream)
    b = lm.embedding_grad(d_out, ids, V)
    torch.cuda.synchronize()
    assert torch.equal(a, first) and torch.equal(b, first) and torch.equal(c, W[ids.long()])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = lm.embedding(ids, W)
        grad = lm.embedding_grad(d_out, ids, V)
    for pattern in ("spread", "none", "one"):
        ids.copy_(draw_ids(pattern, tokens, V, seed=9))
        graph.replay()
        check_status()
        want, tol = ref.embedding_grad(d_out, ids, V)
        assert_close(grad, want, tol, pattern)
        want, tol = ref.embedding(ids, W)
        assert_close(out, want, tol, pattern)


def test_nothing_else_is_written():
    tokens, H, V = 600, 72, 90
    ids, d_out = draw_ids("absent", tokens, V), normal(1, tokens, H)
    whole = torch.full((V * H + 512,), 77.0, dtype=torch.bfloat16, device="cuda")
    need = lm.embedding_grad_workspace_bytes(tokens, V, H)
    ws = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    lm.embedding_grad(d_out, ids, V, out=whole[256:256 + V * H].view(V, H),
                      workspace=ws[256:256 + need])
    check_status()
    for t in (whole, ws):
        assert (t[:256] == 77).all() and (t[-256:] == 77).all()
    want, tol = ref.embedding_grad(d_out, ids, V)
    assert_close(whole[256:256 + V * H].view(V, H), want, tol, "grad")
