"""The training operators around the LM head, as they are measured: the softmax cross entropy over the
vocabulary with its gradient (no logits kept), and the token embedding with its gradient.

With z[r, v] = alpha * (hidden[r] . W[v] + bias[v]) in fp32 and t_r the target of row r,

    lse_r  = log sum_v exp z[r, v]
    loss_r = lse_r - z[r, t_r] + z_loss * lse_r^2          (0 for a row whose target is ignored)
    loss   = sum_r loss_r / (number of rows not ignored), their sum, or the rows themselves
    dz     = g_r * ((1 + 2 z_loss lse_r) * exp(z - lse_r) - [v = t_r])
    d_hidden = alpha * dz @ W,   d_W = alpha * dz^T @ hidden,   d_bias = alpha * sum_r dz

and, for token ids i_t,

    out[t]  = scale * W[i_t]                               (0 for an id outside the table)
    d_W[v]  = scale * sum over {t : i_t = v} of d_out[t]

A case's "op" names the pass: "loss" (a forward pass, as in evaluation), "step" (the loss and its
gradients), "embed" and "embed_grad". Rows of ignored targets hold whatever padding left there
(NaN and infinities among it); no such value may reach a result.
"""
import math

import torch

own = False

IGNORE = -100
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # evaluation of a single next token on a small table: a latency-bound call
        _xent("loss: one row", "loss", 1, 256, 1024, alpha=0.25, reduction="none"),
        # one sequence of per-token scores over the decode head's table
        _xent("loss: 128 rows", "loss", 128, 2048, 151936, reduction="none", masked=0.0),
        # an evaluation batch: forward only, a padded batch with prompts that do not count
        _xent("loss: 8192 rows, masked", "loss", 8192, 2048, 151936, masked=0.25, reduction="mean"),
        # the smallest training step (unit tests, tiny models)
        _xent("step: 32 rows", "step", 32, 256, 1024, alpha=0.25, reduction="mean"),
        # a micro-batch of a few sequences' last tokens with per-row weights (policy gradients)
        _xent("step: 96 rows, weighted", "step", 96, 2048, 151936, reduction="none", masked=0.25),
        # odd sizes, fp16 with a loss scale, an embedding bias and the logit regulariser
        _xent("step: odd sizes, fp16", "step", 777, 1032, 32771, dtype="f16", bias=True, z_loss=1e-4,
              masked=0.1, reduction="mean", grad=1024.0),
        # instruction tuning: most of the batch is prompt or padding
        _xent("step: 4096 rows, mostly masked", "step", 4096, 2048, 151936, masked=0.6, reduction="mean", bias=True),
        # pre-training: every row counts
        _xent("step: 4096 rows", "step", 4096, 4096, 128256, reduction="mean", z_loss=1e-4),
        # decoding: one token's embedding
        _emb("embed: one token", "embed", 1, 2048, 151936),
        # a training batch's embeddings, padded
        _emb("embed: 16384 tokens", "embed", 16384, 4096, 151936, pad=0.05, scale=64.0),
        # small and ragged, with an id that fills half the batch
        _emb("embed_grad: odd sizes", "embed_grad", 1025, 264, 5003, dtype="f16", heavy=0.5, scale=16.25),
        # the gradient of a training batch over a whole table
        _emb("embed_grad: 16384 tokens", "embed_grad", 16384, 4096, 151936, pad=0.05, heavy=0.02, scale=64.0),
    ]


def draw(rng):
    def size(low, high, step=1):
        return max(low, int(math.exp(rng.uniform(math.log(low), math.log(high + 1))) / step) * step)

    dtype = rng.choice(["bf16", "bf16", "f16"])
    if rng.random() < 0.6:
        op = rng.choice(["loss", "step", "step"])
        rows, hidden, vocab = size(1, 4096), size(64, 4096, 8), size(500, 151936)
        rows = min(rows, max(1, 2 * 10 ** 12 // (hidden * vocab)))
        return _xent(None, op, rows, hidden, vocab, dtype=dtype, bias=rng.random() < 0.4,
                     alpha=rng.choice([1.0, 1.0, 0.5, 0.125]), z_loss=rng.choice([0.0, 0.0, 1e-4]),
                     masked=rng.choice([-1.0, -1.0, 0.0, round(rng.uniform(0.05, 0.9), 3)]),
                     reduction=rng.choice(["mean", "mean", "sum", "none"]),
                     grad=1024.0 if dtype == "f16" else 1.0)
    op = rng.choice(["embed", "embed_grad", "embed_grad"])
    hidden = size(64, 4096, 8)
    tokens = min(size(1, 65536), 2 ** 26 // hidden)
    return _emb(None, op, tokens, hidden, size(500, 151936), dtype=dtype, pad=rng.choice([0.0, 0.0, 0.05, 0.3]),
                heavy=0.0 if op == "embed" else rng.choice([0.0, 0.02, 0.5, 1.0]), scale=rng.choice([1.0, 8.0, 45.25]))


def _xent(name, op, rows, hidden, vocab, dtype="bf16", alpha=1.0, bias=False, masked=-1.0, z_loss=0.0, reduction="mean", grad=1.0):
    """masked: the share of rows whose target is ignored; below 0 the call knows of no ignored target."""
    c = {"name": name} if name else {}
    return c | {"op": op, "rows": rows, "hidden": hidden, "vocab": vocab, "dtype": dtype, "alpha": alpha, "bias": bias,
                "masked": masked, "z_loss": z_loss, "reduction": reduction, "grad": grad}


def _emb(name, op, tokens, hidden, vocab, dtype="bf16", pad=0.0, heavy=0.0, scale=1.0):
    """pad: the share of tokens without an id; heavy: the share of tokens that are one and the same id."""
    c = {"name": name} if name else {}
    return c | {"op": op, "tokens": tokens, "hidden": hidden, "vocab": vocab, "dtype": dtype, "pad": pad, "heavy": heavy, "scale": scale}


def _valid_rows(case):
    return case["rows"] - (int(case["masked"] * case["rows"]) if case["masked"] > 0 else 0)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(shape, generator=g, device="cuda")

    dtype, H, V = DTYPES[case["dtype"]], case["hidden"], case["vocab"]
    if case["op"].startswith("embed"):
        T = case["tokens"]
        # frequent ids are the small ones, as in a table sorted by frequency
        ids = (uniform(T) ** 4 * V).long().clamp_(max=V - 1)
        lot = uniform(T)
        ids = torch.where(lot < case["heavy"], torch.full_like(ids, V // 3), ids)
        ids = torch.where(uniform(T) < case["pad"], torch.full_like(ids, -1), ids).to(torch.int32)
        state = {"case": case, "ids": ids}
        if case["op"] == "embed":
            state["W"] = (normal(V, H) * 0.02).to(dtype)
        else:
            state["d_out"] = (normal(T, H) * 0.02).to(dtype)
        return state
    R = case["rows"]
    # logits of a few units' spread whatever alpha is, and targets that the rows foretell in part
    W = normal(V, H).mul_(0.8 / (math.sqrt(H) * case["alpha"])).to(dtype)
    targets = (uniform(R) ** 2 * V).long().clamp_(max=V - 1)
    foretold = W[targets].float()
    foretold *= (uniform(R, 1) * 12.0 / case["alpha"]) / foretold.square().sum(1, keepdim=True)
    hidden = normal(R, H) + foretold
    n_masked = R - _valid_rows(case)
    if n_masked:
        # sequences one behind another: a prompt at each one's head and padding at its tail
        seqs = min(8, R)
        left = n_masked
        bounds = [R * s // seqs for s in range(seqs + 1)]
        for s, part in enumerate(uniform(seqs).tolist()):
            n = bounds[s + 1] - bounds[s]
            m = min(n, -(-left * n // (R - bounds[s])))
            left -= m
            head = int(part * m)
            targets[bounds[s]:bounds[s] + head] = IGNORE
            targets[bounds[s + 1] - (m - head):bounds[s + 1]] = IGNORE
            hidden[bounds[s + 1] - (m - head):bounds[s + 1], ::3] = float("nan")
            hidden[bounds[s + 1] - (m - head):bounds[s + 1], 1::3] = float("inf")
    state = {"case": case, "hidden": hidden.to(dtype), "W": W, "targets": targets.to(torch.int32),
             "bias": (normal(V) * 0.5).to(dtype) if case["bias"] else None}
    # the gradient of the loss: one number, or one for each row
    state["grad_loss"] = normal(R) * (case["grad"] / R) if case["reduction"] == "none" else torch.full((), case["grad"], device="cuda")
    return state


def run(state):
    op = state["case"]["op"]
    if op == "embed":
        return _own_embed(state) if own else _plain_embed(state)
    if op == "embed_grad":
        return _own_embed_grad(state) if own else _plain_embed_grad(state)
    return _own_xent(state) if own else _plain_xent(state)


def _own_xent(state):
    import fp32_accumulate_lm_b200 as lm
    c = state["case"]
    how = {"alpha": c["alpha"], "bias": state["bias"], "z_loss": c["z_loss"], "reduction": c["reduction"],
           "ignore_index": IGNORE if c["masked"] >= 0 else None}
    loss, lse = lm.cross_entropy_f32(state["hidden"], state["W"], state["targets"], **how)
    out = {"loss": loss, "lse": lse}
    if c["op"] == "step":
        d_hidden, d_W, d_bias = lm.cross_entropy_grad(state["hidden"], state["W"], state["targets"], lse, state["grad_loss"], **how)
        out |= {"d_hidden": d_hidden, "d_W": d_W} | ({"d_bias": d_bias} if c["bias"] else {})
    return out


def _own_embed(state):
    import fp32_accumulate_lm_b200 as lm
    return lm.embedding(state["ids"], state["W"], scale=state["case"]["scale"])


def _own_embed_grad(state):
    import fp32_accumulate_lm_b200 as lm
    return lm.embedding_grad(state["d_out"], state["ids"], state["case"]["vocab"], scale=state["case"]["scale"])


def _plain_xent(state):
    c, W = state["case"], state["W"].float()
    dtype = state["W"].dtype
    counts = state["targets"] != IGNORE
    target = torch.where(counts, state["targets"], 0).long()
    # rows that do not count are taken out before any arithmetic: they may hold NaN
    hidden = torch.where(counts[:, None], state["hidden"].float(), 0.0)
    z = hidden @ W.t()
    if state["bias"] is not None:
        z += state["bias"].float()
    z *= c["alpha"]
    top = z.max(1, keepdim=True).values
    lse = torch.log(torch.exp(z - top).sum(1)) + top[:, 0]
    at_target = z.gather(1, target[:, None])[:, 0]
    rows = torch.where(counts, lse - at_target + c["z_loss"] * lse * lse, 0.0)
    n = counts.sum().clamp(min=1)
    loss = rows if c["reduction"] == "none" else rows.sum() if c["reduction"] == "sum" else rows.sum() / n
    out = {"loss": loss, "lse": torch.where(counts, lse, 0.0)}
    if c["op"] == "loss":
        return out
    g = torch.where(counts, state["grad_loss"] / n if c["reduction"] == "mean" else state["grad_loss"].expand(c["rows"]), 0.0)
    dz = torch.exp(z.sub_(lse[:, None]))
    dz *= (1.0 + 2.0 * c["z_loss"] * lse)[:, None]
    dz[torch.arange(c["rows"], device="cuda"), target] -= 1.0
    dz *= (g * c["alpha"])[:, None]
    out |= {"d_hidden": (dz @ W).to(dtype), "d_W": (dz.t() @ hidden).to(dtype)}
    return out | ({"d_bias": dz.sum(0).to(dtype)} if c["bias"] else {})


def _plain_embed(state):
    ids, W, scale = state["ids"], state["W"], state["case"]["scale"]
    rows = W[ids.clamp(min=0).long()].float() * scale
    return torch.where(((ids >= 0) & (ids < W.shape[0]))[:, None], rows, 0.0).to(W.dtype)


def _plain_embed_grad(state):
    ids, d_out, c = state["ids"], state["d_out"], state["case"]
    held = (ids >= 0) & (ids < c["vocab"])
    d_W = torch.zeros((c["vocab"], c["hidden"]), device="cuda")
    d_W.index_add_(0, torch.where(held, ids, 0).long(), torch.where(held[:, None], d_out.float(), 0.0))
    return (d_W * c["scale"]).to(d_out.dtype)


def work(case):
    H, V = case["hidden"], case["vocab"]
    if case["op"].startswith("embed"):
        T = case["tokens"]
        held = T * (1.0 - case["pad"])
        if case["op"] == "embed":
            return {"bytes": 4 * T + 2 * H * (T + held), "flops": H * held}
        return {"bytes": 4 * T + 2 * H * (V + held), "flops": H * held}
    R, n = case["rows"], _valid_rows(case)
    table = 2 * V * H + (2 * V if case["bias"] else 0)
    if case["op"] == "loss":
        return {"bytes": table + 2 * n * H + 12 * R, "flops": 2 * n * V * H}
    # the loss needs the logits once; its gradients need them again (they are not kept) and two products
    return {"bytes": 2 * table + 2 * H * (n + R) + 20 * R, "flops": 8 * n * V * H}


def exact(case, seed):
    """The same outputs in 64 bits, row by row of the definitions: no logits of ignored rows, the
    softmax of torch, the gradients through the centred logits in pieces of the vocabulary."""
    s = prepare(case, seed)
    if case["op"] == "embed":
        out = torch.zeros((case["tokens"], case["hidden"]), dtype=torch.float64, device="cuda")
        at = (s["ids"] >= 0).nonzero()[:, 0]
        out[at] = s["W"].index_select(0, s["ids"][at].long()).double().mul_(case["scale"])
        return out
    if case["op"] == "embed_grad":
        at = (s["ids"] >= 0).nonzero()[:, 0]
        order = at[torch.sort(s["ids"][at], stable=True).indices]
        ids, counts = torch.unique_consecutive(s["ids"][order], return_counts=True)
        ends = counts.cumsum(0)
        sums = torch.cat([torch.zeros((1, case["hidden"]), dtype=torch.float64, device="cuda"),
                          s["d_out"][order].double().cumsum(0)])
        d_W = torch.zeros((case["vocab"], case["hidden"]), dtype=torch.float64, device="cuda")
        d_W[ids.long()] = (sums[ends] - sums[ends - counts]) * case["scale"]
        return d_W
    R, V = case["rows"], case["vocab"]
    rows = (s["targets"] != IGNORE).nonzero()[:, 0]
    h, t = s["hidden"][rows].double(), s["targets"][rows].long()
    W = s["W"].double()
    z = torch.mm(h, W.t()).mul_(case["alpha"])
    if case["bias"]:
        z += s["bias"].double() * case["alpha"]
    lse = torch.logsumexp(z, 1) if rows.numel() else z.new_zeros(0)
    each = lse - z[torch.arange(rows.numel(), device="cuda"), t] + case["z_loss"] * lse ** 2

    def spread(x):
        whole = torch.zeros((R, *x.shape[1:]), dtype=torch.float64, device="cuda")
        whole[rows] = x
        return whole

    n = max(rows.numel(), 1)
    loss = spread(each) if case["reduction"] == "none" else each.sum() / (n if case["reduction"] == "mean" else 1)
    out = {"loss": loss, "lse": spread(lse)}
    if case["op"] == "loss":
        return out
    up = s["grad_loss"].double()
    up = up[rows] if case["reduction"] == "none" else (up / (n if case["reduction"] == "mean" else 1)).expand(rows.numel())
    up = up * case["alpha"]
    d_h, d_W = torch.zeros_like(h), torch.zeros_like(W)
    d_b = torch.zeros(V, dtype=torch.float64, device="cuda")
    factor = (up * (1.0 + 2.0 * case["z_loss"] * lse))[:, None]
    for v in range(0, V, 16384):
        piece = torch.exp(z[:, v:v + 16384] - lse[:, None]) * factor
        hit = ((t >= v) & (t < v + 16384)).nonzero()[:, 0]
        piece[hit, t[hit] - v] -= up[hit]
        d_h.addmm_(piece, W[v:v + 16384])
        d_W[v:v + 16384] = piece.t() @ h
        d_b[v:v + 16384] = piece.sum(0)
    out |= {"d_hidden": spread(d_h), "d_W": d_W}
    return out | ({"d_bias": d_b} if case["bias"] else {})
