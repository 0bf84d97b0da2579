"""The operators at a model's two ends and between its blocks, as measured cases.

Three operators: the embedding lookup with scaling and an addend, and its
gradient by sorted tokens; dropout from a counter-based generator with the
residual's addition (its gradient is the same call without a residual); and the
softmax cross entropy of a projection onto a large vocabulary, with its
gradients, where the logits are never kept.

Each case runs in two forms on the same inputs: `own` false, elementary torch
operations in 32 bits; `own` true, this package's entry points. `exact` gives
the values of the definitions in 64 bits.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
SIZES = {"bf16": 2, "f32": 4}
MASK32 = 0xFFFFFFFF
# Philox4x32 (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3", 2011)
MULTIPLIERS = (0xD2511F53, 0xCD9E8D57)
WEYL = (0x9E3779B9, 0xBB67AE85)
ROUNDS = 10


def listed():
    return [
        # one token's row: the first call of a decoding step
        _embed("embed_one_token", 1, 4096, 32000, "bf16", "i64", False),
        # a GPT-2 batch, tokens' rows added to the positions'
        _embed("embed_gpt2_addend", 8192, 768, 50257, "bf16", "i64", True),
        # the Llama root unit's table: eight ranks' 2048 tokens
        _embed("embed_llama", 16384, 4096, 32000, "bf16", "i64", False),
        # a small fp32 model of odd width
        _embed_bwd("embed_bwd_odd", 333, 769, 1009, "f32", "f32", "i64", False),
        # GPT-2's tied table: added to the gradient that the head has left
        _embed_bwd("embed_bwd_gpt2_tied", 8192, 768, 50257, "bf16", "bf16", "i64", True),
        # the Llama root unit's table, its whole gradient written
        _embed_bwd("embed_bwd_llama", 16384, 4096, 32000, "bf16", "bf16", "i32", False),
        # a short odd batch
        _dropout("dropout_odd", 33, 769, "f32", False, 0.1),
        # a block's output added to the residual stream in training
        _dropout("dropout_block", 16384, 4096, "bf16", True, 0.1),
        # a tiny model: latency
        _ce("ce_tiny", 37, 64, 1000, 0.1, "all", False),
        # evaluation of one sequence: losses alone
        _ce("ce_llama_eval", 511, 4096, 32000, 0.0, "loss", False),
        # one rank's batch through GPT-2's head (odd vocabulary)
        _ce("ce_gpt2", 8192, 768, 50257, 0.02, "all", False),
        # one rank's batch through the Llama head, each token's loss with a weight of its own
        _ce("ce_llama", 4096, 4096, 32000, 0.05, "all", True),
    ]


def _embed(name, rows, cols, vocab, dtype, index, addend):
    return _named(name, {"op": "embed", "rows": rows, "cols": cols, "vocab": vocab, "dtype": dtype, "index": index,
                         "addend": addend})


def _embed_bwd(name, rows, cols, vocab, dtype, table, index, accumulate):
    return _named(name, {"op": "embed_bwd", "rows": rows, "cols": cols, "vocab": vocab, "dtype": dtype, "table": table,
                         "index": index, "accumulate": accumulate})


def _dropout(name, rows, cols, dtype, residual, p):
    return _named(name, {"op": "dropout", "rows": rows, "cols": cols, "dtype": dtype, "residual": residual, "p": p})


def _ce(name, rows, cols, vocab, without, outputs, weighted):
    return _named(name, {"op": "ce", "rows": rows, "cols": cols, "vocab": vocab, "without": without,
                         "outputs": outputs, "weighted": weighted})


def _named(name, case):
    return dict(case, name=name) if name else case


def draw(rng):
    def spread(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))))

    op = rng.choice(["embed", "embed_bwd", "embed_bwd", "dropout", "ce", "ce", "ce"])
    if op == "dropout":
        cols = rng.choice([768, 4096, spread(1, 16384), spread(1, 16384)])
        rows = spread(1, min(65536, 16384 * 4096 // cols))
        return _dropout(None, rows, cols, rng.choice(["bf16", "bf16", "f32"]), rng.random() < 0.6,
                        rng.choice([0.0, 0.1, 0.5, 0.05 + 0.9 * rng.random()]))
    vocab = rng.choice([32000, 50257, spread(2, 131072), spread(2, 131072)])
    if op == "ce":
        cols = rng.choice([64, 768, 4096, spread(1, 4096), spread(8, 4096)])
        vocab = min(vocab, 65536)
        rows = spread(1, min(16384, 4096 * 4096 * 32000 // (cols * vocab)))
        outputs = rng.choice(["all", "all", "loss"])
        return _ce(None, rows, cols, vocab, rng.choice([0.0, 0.02, 0.3]), outputs, outputs == "all" and rng.random() < 0.4)
    cols = rng.choice([768, 4096, spread(1, 8192), spread(1, 8192)])
    vocab = min(vocab, 32000 * 4096 // cols)
    rows = spread(1, min(131072, 16384 * 4096 // cols))
    dtype, index = rng.choice(["bf16", "bf16", "f32"]), rng.choice(["i64", "i64", "i32"])
    if op == "embed":
        return _embed(None, rows, cols, vocab, dtype, index, rng.random() < 0.4)
    return _embed_bwd(None, rows, cols, vocab, dtype, rng.choice([dtype, dtype, "bf16", "f32"]), index,
                      rng.random() < 0.4)


def work(case):
    rows, cols, op = case["rows"], case["cols"], case["op"]
    n = rows * cols
    if op == "dropout":
        e = SIZES[case["dtype"]]
        return {"bytes": n * e * (3 if case["residual"] else 2), "flops": 3 * n}
    vocab = case["vocab"]
    if op == "ce":
        weight = vocab * cols
        given = 2 * (n + weight) + 8 * rows + (4 * rows if case["weighted"] else 0) + 8 * rows
        if case["outputs"] == "loss":
            return {"bytes": given, "flops": 2 * rows * weight}
        return {"bytes": given + 2 * (n + weight), "flops": 6 * rows * weight}
    e, index = SIZES[case["dtype"]], 8 if case["index"] == "i64" else 4
    touched = _distinct(rows, vocab) * cols  # table rows that some token names
    if op == "embed":
        return {"bytes": touched * e + n * e * (2 if case["addend"] else 1) + rows * index,
                "flops": n * (2 if case["addend"] else 1)}
    t = SIZES[case["table"]]
    table = 2 * touched * t if case["accumulate"] else vocab * cols * t
    return {"bytes": n * e + rows * index + table, "flops": n}


def _distinct(rows, vocab):
    """About how many different tokens `rows` draws of prepare()'s distribution give (token of rank k: 1 / k)."""
    k = np.arange(1, vocab + 1)
    share = np.log((k + 1) / k) / math.log(vocab + 1)
    return int(round(float((1 - (1 - share) ** rows).sum())))


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=gen, device="cuda")

    def tokens(rows, vocab):
        # a text's: the k-th most frequent one has a share of about 1 / k
        rank = (torch.exp(uniform(rows).double() * math.log(vocab + 1)) - 1).long().clamp(0, vocab - 1)
        return torch.randperm(vocab, generator=gen, device="cuda")[rank]

    state = dict(case)
    rows, cols, op = case["rows"], case["cols"], case["op"]
    if op == "dropout":
        dtype = DTYPES[case["dtype"]]
        state["x"] = normal(rows, cols).to(dtype)
        state["residual"] = (4 * normal(rows, cols)).to(dtype) if case["residual"] else None
        state["out"] = torch.empty(rows, cols, dtype=dtype, device="cuda")
        state["seed"] = (seed * 0x9E3779B97F4A7C15 + 1) & (2 ** 63 - 1)
        state["offset"] = seed * 1009 + 17
        return state

    vocab = case["vocab"]
    if op == "ce":
        # a model in training: rows of unit size, the target's logit raised by very different amounts
        weight = (normal(vocab, cols) / math.sqrt(cols)).to(torch.bfloat16)
        targets = tokens(rows, vocab)
        hidden = normal(rows, cols) + (10 * uniform(rows))[:, None] * weight[targets].float()
        state["hidden"], state["weight"] = hidden.to(torch.bfloat16), weight
        state["targets"] = torch.where(uniform(rows) < case["without"], -100, targets)
        state["loss"], state["lse"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        if case["outputs"] == "all":
            state["dhidden"], state["dweight"] = torch.empty_like(state["hidden"]), torch.empty_like(weight)
            state["dloss"] = 0.5 + uniform(rows) if case["weighted"] else None
            state["scale"] = 1.0 / rows
        return state

    index = torch.int64 if case["index"] == "i64" else torch.int32
    ids = tokens(rows, vocab)
    dtype = DTYPES[case["dtype"]]
    if op == "embed":
        state["tokens"] = ids.to(index)
        state["table"] = (0.02 * normal(vocab, cols)).to(dtype)
        state["addend"] = (0.02 * normal(rows, cols)).to(dtype) if case["addend"] else None
        state["out"] = torch.empty(rows, cols, dtype=dtype, device="cuda")
        state["scale"] = 1.0 if case["addend"] else math.sqrt(cols)
        return state
    state["tokens"] = torch.where(uniform(rows) < 0.02, -1, ids).to(index)  # some rows are padding
    state["dout"] = (1e-3 * normal(rows, cols)).to(dtype)
    state["dtable"] = (1e-3 * normal(vocab, cols)).to(DTYPES[case["table"]])
    state["scale"] = 1.0 if case["accumulate"] else math.sqrt(cols)
    return state


# --------------------------------------------------------------- the passes


def run(state):
    return (_run_own if own else _run_plain)[state["op"]](state)


def _plain_embed(s):
    out = s["scale"] * s["table"][s["tokens"]].float()
    if s["addend"] is not None:
        out = out + s["addend"].float()
    return {"out": out.to(s["out"].dtype)}


def _own_embed(s):
    import fully_sharded_gb300 as fs

    fs.fsdp_embedding(s["tokens"], s["table"], s["out"], scale=s["scale"], addend=s["addend"])
    return {"out": s["out"]}


def _plain_embed_bwd(s):
    there = s["tokens"] >= 0
    rows = torch.where(there[:, None], s["scale"] * s["dout"].float(), 0.0)
    base = s["dtable"].float() if s["accumulate"] else torch.zeros(s["vocab"], s["cols"], device="cuda")
    base.index_add_(0, s["tokens"].clamp(min=0), rows)
    s["dtable"].copy_(base)
    return {"dtable": s["dtable"]}


def _own_embed_bwd(s):
    import fully_sharded_gb300 as fs

    if "workspace" not in s:  # kept as a training loop keeps it
        s["workspace"] = _bytes(fs.fsdp_embedding_backward_workspace(s["rows"], s["cols"], s["vocab"]))
    fs.fsdp_embedding_backward(s["tokens"], s["dout"], s["dtable"], s["workspace"], scale=s["scale"],
                               accumulate=s["accumulate"])
    return {"dtable": s["dtable"]}


def _philox(counter, seed, offset):
    """Four 32-bit words for each of the 64-bit counters, as int64."""
    c = [counter & MASK32, counter >> 32 & MASK32, torch.full_like(counter, offset & MASK32),
         torch.full_like(counter, offset >> 32 & MASK32)]
    k0, k1 = seed & MASK32, seed >> 32 & MASK32
    a, b = MULTIPLIERS
    for _ in range(ROUNDS):
        p0, p1 = a * c[0], b * c[2]  # modulo 2^64, which keeps both halves
        c = [(p1 >> 32 & MASK32) ^ c[1] ^ k0, p1 & MASK32, (p0 >> 32 & MASK32) ^ c[3] ^ k1, p0 & MASK32]
        k0, k1 = (k0 + WEYL[0]) & MASK32, (k1 + WEYL[1]) & MASK32
    return c


def _plain_dropout(s):
    rows, cols = s["rows"], s["cols"]
    threshold = math.floor(s["p"] * 65536 + 0.5)
    words = _philox(torch.arange(-(-rows * cols // 8), device="cuda"), s["seed"], s["offset"])
    draws = torch.stack([half for w in words for half in (w & 0xFFFF, w >> 16)], 1)  # 8 draws of 16 bits a counter
    keep = (draws.reshape(-1)[:rows * cols] >= threshold).view(rows, cols)
    out = torch.where(keep, s["x"].float() * (65536.0 / (65536 - threshold)), 0.0)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return {"out": out.to(s["x"].dtype)}


def _own_dropout(s):
    import fully_sharded_gb300 as fs

    fs.fsdp_dropout(s["x"], s["out"], s["p"], s["seed"], s["offset"], residual=s["residual"])
    return {"out": s["out"]}


def _plain_ce(s):
    hidden, weight, targets = s["hidden"].float(), s["weight"].float(), s["targets"]
    there, at = targets >= 0, targets.clamp(min=0)[:, None]
    logits = hidden @ weight.t()
    most = logits.amax(1)
    lse = most + torch.log(torch.exp(logits - most[:, None]).sum(1))
    out = {"loss": torch.where(there, lse - logits.gather(1, at)[:, 0], 0.0), "lse": lse}
    if s["outputs"] == "all":
        factor = s["scale"] * (s["dloss"] if s["dloss"] is not None else torch.ones_like(lse))
        g = torch.exp(logits - lse[:, None])
        g.scatter_add_(1, at, torch.full_like(at, -1, dtype=g.dtype))
        g = g * torch.where(there, factor, 0.0)[:, None]
        out["dhidden"] = (g @ weight).to(torch.bfloat16)
        out["dweight"] = (g.t() @ hidden).to(torch.bfloat16)
    return out


def _own_ce(s):
    import fully_sharded_gb300 as fs

    every = s["outputs"] == "all"
    if "workspace" not in s:  # kept as a training loop keeps it
        s["workspace"] = _bytes(fs.fsdp_cross_entropy_workspace(s["rows"], s["cols"], s["vocab"], gradients=every))
    if not every:
        fs.fsdp_cross_entropy(s["hidden"], s["weight"], s["targets"], s["loss"], s["workspace"], lse=s["lse"])
        return {"loss": s["loss"], "lse": s["lse"]}
    fs.fsdp_cross_entropy(s["hidden"], s["weight"], s["targets"], s["loss"], s["workspace"], lse=s["lse"],
                          dhidden=s["dhidden"], dweight=s["dweight"], scale=s["scale"], dloss=s["dloss"])
    return {k: s[k] for k in ("loss", "lse", "dhidden", "dweight")}


def _bytes(n):
    return torch.empty(max(1, n), dtype=torch.uint8, device="cuda")


_run_plain = {"embed": _plain_embed, "embed_bwd": _plain_embed_bwd, "dropout": _plain_dropout, "ce": _plain_ce}
_run_own = {"embed": _own_embed, "embed_bwd": _own_embed_bwd, "dropout": _own_dropout, "ce": _own_ce}


# ------------------------------------------------------- the 64-bit values


def exact(case, seed):
    s = prepare(case, seed)
    return {"embed": _exact_embed, "embed_bwd": _exact_embed_bwd, "dropout": _exact_dropout, "ce": _exact_ce}[case["op"]](s)


def _exact_embed(s):
    out = torch.index_select(s["table"], 0, s["tokens"]).double().mul_(s["scale"])
    return {"out": out if s["addend"] is None else out.add_(s["addend"])}


def _exact_embed_bwd(s):
    """Sums over the sorted tokens, as differences of the running sums of each span of columns."""
    ids, order = torch.sort(s["tokens"].long(), stable=True)
    first = int((ids < 0).sum())
    ids, order = ids[first:], order[first:]
    bounds = torch.searchsorted(ids, torch.arange(s["vocab"] + 1, device="cuda"))
    out = s["dtable"].double() if s["accumulate"] else torch.zeros(s["vocab"], s["cols"], dtype=torch.float64, device="cuda")
    for c in range(0, s["cols"], 512):
        span = s["dout"][order, c:c + 512].double()
        running = torch.cat([span.new_zeros(1, span.shape[1]), span.cumsum(0)])
        out[:, c:c + 512] += s["scale"] * (running[bounds[1:]] - running[bounds[:-1]])
    return {"dtable": out}


def _exact_dropout(s):
    rows, cols, u = s["rows"], s["cols"], np.uint64
    n = rows * cols
    mask, shift = u(MASK32), u(32)
    lanes = np.empty((-(-n // 8), 8), dtype=np.uint16)
    for at in range(0, len(lanes), 1 << 20):
        x0 = np.arange(at, min(len(lanes), at + (1 << 20)), dtype=u)
        x1, x0 = x0 >> shift, x0 & mask
        x2, x3 = np.full_like(x0, s["offset"] & MASK32), np.full_like(x0, s["offset"] >> 32)
        key = [s["seed"] & MASK32, s["seed"] >> 32]
        for _ in range(ROUNDS):
            lo, hi = x0 * u(MULTIPLIERS[0]), x2 * u(MULTIPLIERS[1])
            x0, x1, x2, x3 = (hi >> shift) ^ x1 ^ u(key[0]), hi & mask, (lo >> shift) ^ x3 ^ u(key[1]), lo & mask
            key = [(k + w) & MASK32 for k, w in zip(key, WEYL)]
        words = np.stack([x0, x1, x2, x3], 1).astype("<u4")
        lanes[at:at + len(words)] = words.view("<u2")
    bound = int(round(s["p"] * 2 ** 16 + 1e-12))
    dropped = torch.from_numpy((lanes.reshape(-1)[:n] < bound).reshape(rows, cols)).cuda()
    out = (s["x"].double() / (1 - bound / 2 ** 16)).masked_fill_(dropped, 0)
    return {"out": out if s["residual"] is None else out + s["residual"].double()}


def _exact_ce(s):
    if 6 * s["rows"] * s["cols"] * s["vocab"] > 8e12:
        return None  # many seconds of 64-bit products
    weight = s["weight"].double()
    out = {k: [] for k in ("loss", "lse", "dhidden")}
    total = torch.zeros_like(weight) if s["outputs"] == "all" else None
    for at in range(0, s["rows"], 1024):  # rows are independent of one another
        hidden, targets = s["hidden"][at:at + 1024].double(), s["targets"][at:at + 1024]
        score = torch.einsum("rc,vc->rv", hidden, weight)
        lse = torch.logsumexp(score, 1)
        some = torch.nonzero(targets >= 0)[:, 0]
        loss = torch.zeros_like(lse)
        loss[some] = lse[some] - score[some, targets[some]]
        out["loss"].append(loss), out["lse"].append(lse)
        if total is None:
            continue
        share = torch.zeros_like(lse)
        share[some] = s["scale"]
        if s["dloss"] is not None:
            share *= s["dloss"][at:at + 1024]
        p = score.sub_(lse[:, None]).exp_()
        p[some, targets[some]] -= 1
        p *= share[:, None]
        out["dhidden"].append(p @ weight)
        total += p.mT @ hidden
    out = {k: torch.cat(v) for k, v in out.items() if v}
    if total is not None:
        out["dweight"] = total
    return out
