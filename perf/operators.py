"""The training operators around a FlatParameter step, as measured cases.

Three operators: RMS norm with the residual's addition (forward, with 8-bit
outputs, and backward), the Newton-Schulz orthogonalisation of update
matrices, and the Muon step of an FSDP unit (reduce-scatter, momentum,
orthogonalisation, master update, cast and gather in one call).

Each case runs in two forms on the same inputs: `own` false, elementary torch
operations in 32 bits; `own` true, this package's entry points. `exact` gives
the values of the definitions in 64 bits.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -126
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "e4m3": torch.float8_e4m3fn}
SIZES = {"bf16": 2, "f32": 4, "e4m3": 1}

# Unit shapes of the package's own workloads: the tiny MLP, one GPT-2 block, one Llama-style block.
TINY_MLP = "64x32,32,32x16,16"
GPT2_BLOCK = "768,768,768x2304,2304,768x768,768,768,768,768x3072,3072,3072x768,768"
LLAMA_BLOCK = "4096x4096,4096x4096,4096x4096,4096x4096,11008x4096,11008x4096,4096x11008,4096,4096"


def listed():
    return [
        # one token's step through the block's norm, its output quantised for an 8-bit product
        _norm("norm_one_token", 1, 4096, "bf16", True, "e4m3", 0),
        # the block's norm in training: eight ranks' 2048 tokens
        _norm("norm_block", 16384, 4096, "bf16", True, "bf16", 0),
        # the wide activation before the down projection, in 8 bits with a scale per 128 values; odd row count
        _norm("norm_8bit_groups", 4097, 11008, "bf16", False, "e4m3", 128),
        # a small fp32 model with an odd width: rows off vector alignment
        _norm_bwd("norm_bwd_odd", 333, 769, "f32", False, "f32"),
        # the block's norm in the backward pass, with the gradient that flows along the residual
        _norm_bwd("norm_bwd_block", 16384, 4096, "bf16", True, "bf16"),
        # the tiny MLP's two matrices: pure latency
        _ns("ns_tiny_mlp", "64x32,32x16", "f32", 0),
        # the four matrices of a GPT-2 block, together
        _ns("ns_gpt2_block", "768x2304,768x768,768x3072,3072x768", "bf16", 0),
        # an odd matrix, read out of a wider buffer
        _ns("ns_odd_strided", "1537x769", "f32", 7),
        # the Llama block's down projection: one large matrix
        _ns("ns_llama_down", "4096x11008", "f32", 0),
        # whole units: the smallest, an ordinary and the largest one of the package's workloads
        _muon("muon_tiny_mlp", TINY_MLP, 4, True, 0.0),
        _muon("muon_gpt2_block", GPT2_BLOCK, 8, True, 0.1),
        _muon("muon_llama_block", LLAMA_BLOCK, 8, True, 0.1),
    ]


def _norm(name, rows, cols, dtype, residual, out, group):
    return _named(name, {"op": "norm", "rows": rows, "cols": cols, "dtype": dtype, "residual": residual, "out": out,
                         "group": group})


def _norm_bwd(name, rows, cols, dtype, residual, gain):
    return _named(name, {"op": "norm_bwd", "rows": rows, "cols": cols, "dtype": dtype, "residual": residual,
                         "gain": gain})


def _ns(name, shapes, dtype, pad):
    return _named(name, {"op": "ns", "shapes": shapes, "dtype": dtype, "pad": pad})


def _muon(name, shapes, world, nesterov, decay):
    return _named(name, {"op": "muon", "shapes": shapes, "world": world, "nesterov": nesterov, "decay": decay})


def _named(name, case):
    return dict(case, name=name) if name else case


def draw(rng):
    def spread(lo, hi):
        return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["norm", "norm", "norm_bwd", "ns", "ns", "muon"])
    if op in ("norm", "norm_bwd"):
        cols = rng.choice([768, 4096, 11008, spread(1, 16384), spread(1, 16384)])
        rows = spread(1, min(65536, max(1, 16384 * 4096 // cols)))
        dtype = rng.choice(["bf16", "bf16", "f32"])
        residual = rng.random() < 0.6
        if op == "norm":
            out = rng.choice([dtype, dtype, "e4m3"])
            group = rng.choice([0, 32, 64, 128, 256]) if out == "e4m3" else 0
            return _norm(None, rows, cols, dtype, residual, out, group)
        return _norm_bwd(None, rows, cols, dtype, residual, rng.choice(["bf16", "f32"]))
    if op == "ns":
        top = rng.choice([64, 512, 4096])
        shapes = ["%dx%d" % (spread(1, top), spread(1, top)) for _ in range(rng.randint(1, 4))]
        return _ns(None, ",".join(shapes), rng.choice(["bf16", "f32"]), rng.choice([0, 0, 1, 8]))
    top = rng.choice([64, 512, 2048])
    shapes = ["%dx%d" % (spread(2, top), spread(2, top)) for _ in range(rng.randint(1, 4))]
    for _ in range(rng.randint(0, 4)):
        shapes.insert(rng.randint(0, len(shapes)), "%d" % spread(1, 4096))
    return _muon(None, ",".join(shapes), rng.choice([1, 2, 3, 4, 8, 8, 16]), rng.random() < 0.7, rng.choice([0.0, 0.1]))


def _shapes(text):
    return [tuple(int(d) for d in part.split("x")) for part in text.split(",")]


def _groups(case):
    return -(-case["cols"] // case["group"]) if case["group"] else 1


def _ns_flops(shapes, steps=5):
    total = 0
    for shape in shapes:
        if len(shape) == 2:
            r, c = min(shape), max(shape)
            total += steps * (r * (r + 1) * c + r * r * (r + 1) + 2 * r * r * c)  # two symmetric products, one full
    return total


def work(case):
    op = case["op"]
    if op == "norm":
        n, e, o = case["rows"] * case["cols"], SIZES[case["dtype"]], SIZES[case["out"]]
        scales = 4 * case["rows"] * _groups(case) if case["out"] == "e4m3" else 0
        return {"bytes": n * (e + o + (2 * e if case["residual"] else 0)) + 4 * case["rows"] + e * case["cols"] + scales,
                "flops": 5 * n}
    if op == "norm_bwd":
        n, e, g = case["rows"] * case["cols"], SIZES[case["dtype"]], SIZES[case["gain"]]
        return {"bytes": n * e * (4 if case["residual"] else 3) + 4 * case["rows"] + 2 * g * case["cols"], "flops": 10 * n}
    shapes = _shapes(case["shapes"])
    if op == "ns":
        return {"bytes": sum(a * b for a, b in shapes) * (SIZES[case["dtype"]] + 2), "flops": _ns_flops(shapes)}
    matrices = sum(math.prod(s) for s in shapes if len(s) == 2)
    others = sum(math.prod(s) for s in shapes if len(s) == 1)
    # gradients, momentum and master read, momentum, master and parameters written (Adam: one more state)
    return {"bytes": matrices * (2 * case["world"] + 18) + others * (2 * case["world"] + 26),
            "flops": _ns_flops(shapes) + matrices * (case["world"] + 8) + others * (case["world"] + 15)}


# ------------------------------------------------------------------ inputs


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=dtype)

    state = dict(case)
    op = case["op"]
    if op in ("norm", "norm_bwd"):
        rows, cols, dtype = case["rows"], case["cols"], DTYPES[case["dtype"]]
        # a residual stream: some channels are much larger than the others
        channel = torch.exp(0.5 * normal(cols))
        state["eps"] = 1e-6
        if op == "norm":
            state["x"] = normal(rows, cols).to(dtype)
            state["residual"] = (normal(rows, cols) * channel).to(dtype) if case["residual"] else None
            state["gain"] = (1 + 0.2 * normal(cols)).to(dtype)
            state["y"] = torch.empty(rows, cols, dtype=DTYPES[case["out"]], device="cuda")
            state["h_out"] = torch.empty(rows, cols, dtype=dtype, device="cuda") if case["residual"] else None
            state["scales"] = torch.empty(rows, _groups(case), device="cuda") if case["out"] == "e4m3" else None
            state["rstd"] = torch.empty(rows, device="cuda")
            return state
        state["h"] = (normal(rows, cols) * channel).to(dtype)
        state["rstd"] = (state["h"].double().square().mean(1) + state["eps"]).rsqrt().float()
        state["dy"] = (1e-3 * normal(rows, cols)).to(dtype)
        state["dh"] = (1e-3 * normal(rows, cols)).to(dtype) if case["residual"] else None
        gain_dtype = DTYPES[case["gain"]]
        state["gain"] = (1 + 0.2 * normal(cols)).to(gain_dtype)
        state["dx"] = torch.empty(rows, cols, dtype=dtype, device="cuda")
        state["dgain"] = torch.empty(cols, dtype=gain_dtype, device="cuda")
        return state

    shapes = _shapes(case["shapes"])

    def gradient(rows, cols):
        # a few strong directions over noise, as an accumulated gradient has
        k = max(1, min(rows, cols) // 16)
        strength = torch.arange(1, k + 1, device="cuda", dtype=torch.float32) ** -0.5
        return 1e-3 * (normal(rows, cols) + (normal(rows, k) * strength) @ normal(k, cols))

    if op == "ns":
        dtype, pad = DTYPES[case["dtype"]], case["pad"]
        state["sources"], state["outs"] = [], []
        for rows, cols in shapes:
            whole = torch.zeros(rows, cols + pad, dtype=dtype, device="cuda")
            whole[:, :cols] = gradient(rows, cols).to(dtype)
            state["sources"].append(whole[:, :cols])
            state["outs"].append(torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda"))
        return state

    world = case["world"]
    numel = sum(math.prod(s) for s in shapes)
    shard = -(-numel // world)
    state.update(numel=numel, shard=shard, lr=2e-4, momentum=0.95, adam_step=10)
    state["grads"] = torch.zeros(world, world * shard, dtype=torch.bfloat16, device="cuda")
    for name, size in (("master", 0.02), ("exp_avg", 0.0), ("exp_avg_sq", 0.0)):
        state[name] = torch.zeros(world * shard, device="cuda")
        if size:
            state[name][:numel] = size * normal(numel)
    at = 0
    for shape in shapes:
        n = math.prod(shape)
        part = gradient(*shape).reshape(-1) if len(shape) == 2 else 1e-3 * normal(n)
        for k in range(world):
            state["grads"][k, at:at + n] = (part + 1e-3 * normal(n)).to(torch.bfloat16)
        state["exp_avg"][at:at + n] = (5.0 if len(shape) == 2 else 0.1) * part + 1e-4 * normal(n)
        if len(shape) == 1:
            state["exp_avg_sq"][at:at + n] = (1e-4 * normal(n)).abs()
        at += n
    state["full_out"] = torch.zeros(world * shard, dtype=torch.bfloat16, device="cuda")
    return state


# --------------------------------------------------------------- the passes


def run(state):
    return (_run_own if own else _run_plain)[state["op"]](state)


def _plain_norm(s):
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    rstd = torch.rsqrt(h.square().mean(1) + s["eps"])
    y = h * rstd[:, None] * s["gain"].float()
    out = {"rstd": rstd}
    if s["residual"] is not None:
        out["h"] = h.to(s["x"].dtype)
    if s["scales"] is None:
        out["y"] = y.to(s["y"].dtype)
        return out
    rows, cols, group = s["rows"], s["cols"], s["group"] or s["cols"]
    padded = torch.nn.functional.pad(y, (0, -cols % group)).view(rows, -1, group)
    scales = (padded.abs().amax(2) / E4M3_MAX).clamp(min=TINY)
    q = (padded / scales[:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).view(rows, -1)[:, :cols]
    out["y"], out["scales"] = q.to(torch.float8_e4m3fn), scales
    return out


def _own_norm(s):
    import fully_sharded_gb300 as fs

    fs.fsdp_rmsnorm(s["x"], s["gain"], s["y"], residual=s["residual"], h_out=s["h_out"], scales=s["scales"],
                    rstd=s["rstd"], group=s["group"], eps=s["eps"])
    out = {"rstd": s["rstd"], "y": s["y"]}
    if s["residual"] is not None:
        out["h"] = s["h_out"]
    if s["scales"] is not None:
        out["scales"] = s["scales"]
    return out


def _plain_norm_bwd(s):
    h, dy, rstd = s["h"].float(), s["dy"].float(), s["rstd"][:, None]
    xhat = h * rstd
    u = dy * s["gain"].float()
    dx = rstd * (u - xhat * (u * xhat).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"dx": dx.to(s["h"].dtype), "dgain": (dy * xhat).sum(0).to(s["gain"].dtype)}


def _own_norm_bwd(s):
    import fully_sharded_gb300 as fs

    if "workspace" not in s:
        s["workspace"] = _bytes(fs.fsdp_rmsnorm_backward_workspace(s["rows"], s["cols"]))
    fs.fsdp_rmsnorm_backward(s["dy"], s["h"], s["gain"], s["rstd"], s["dx"], s["dgain"], s["workspace"], dh=s["dh"])
    return {"dx": s["dx"], "dgain": s["dgain"]}


def _orthogonal(g, dtype):
    x = g.to(dtype)
    if x.shape[0] > x.shape[1]:
        return _orthogonal(g.t(), dtype).t()
    x = x / (x.square().sum().sqrt() + 1e-7)
    a, b, c = COEFFICIENTS
    for _ in range(5):
        gram = x @ x.t()
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x


def _plain_ns(s):
    return [_orthogonal(g, torch.float32).to(torch.bfloat16) for g in s["sources"]]


def _own_ns(s):
    import fully_sharded_gb300 as fs

    if "batch" not in s:  # the prepared call: the matrices' table and a workspace, kept as a training loop keeps them
        s["batch"] = fs.NewtonSchulzBatch(s["sources"], s["outs"])
        s["workspace"] = _bytes(fs.fsdp_newton_schulz_workspace(s["batch"]))
    fs.fsdp_newton_schulz(s["batch"], s["workspace"])
    return s["outs"]


def _scale(rows, cols):
    return 0.2 * math.sqrt(max(rows, cols))  # an update of the size that Adam's has


def _plain_muon(s):
    g = s["grads"].float().sum(0) / s["world"]
    at = 0
    for shape in _shapes(s["shapes"]):
        n = math.prod(shape)
        part = slice(at, at + n)
        at += n
        p, m, v, gp = s["master"][part], s["exp_avg"][part], s["exp_avg_sq"][part], g[part]
        if len(shape) == 2:
            m.mul_(s["momentum"]).add_(gp)
            u = gp + s["momentum"] * m if s["nesterov"] else m
            o = _orthogonal(u.view(shape), torch.float32).reshape(-1)
            p.mul_(1 - s["lr"] * s["decay"]).sub_(s["lr"] * _scale(*shape) * o)
        else:
            m.mul_(0.9).add_(0.1 * gp)
            v.mul_(0.95).add_(0.05 * gp * gp)
            mhat, vhat = m / (1 - 0.9 ** s["adam_step"]), v / (1 - 0.95 ** s["adam_step"])
            p.sub_(s["lr"] * mhat / (vhat.sqrt() + 1e-8))
    s["full_out"].copy_(s["master"])
    return {k: s[k] for k in ("master", "exp_avg", "exp_avg_sq", "full_out")}


def _own_muon(s):
    import fully_sharded_gb300 as fs

    if "unit" not in s:  # the unit's layout, table and workspace, kept as a training loop keeps them
        shapes = _shapes(s["shapes"])
        layout, _ = fs.fsdp_flatten_layout([math.prod(x) for x in shapes], s["world"])
        tensors = [fs.MuonTensor(x[0], x[1], _scale(*x)) if len(x) == 2 else fs.MuonTensor(x[0]) for x in shapes]
        shards = {k: list(s[k].view(s["world"], -1)) for k in ("master", "exp_avg", "exp_avg_sq")}
        s["unit"] = fs.MuonUnit(layout, tensors, list(s["grads"]), full_out=s["full_out"], **shards)
        s["workspace"] = _bytes(fs.fsdp_muon_workspace(s["unit"]))
    muon = fs.Muon(lr=s["lr"], momentum=s["momentum"], nesterov=s["nesterov"], weight_decay=s["decay"],
                   adam=fs.AdamHyper(lr=s["lr"], beta1=0.9, beta2=0.95, eps=1e-8, step=s["adam_step"]))
    fs.fsdp_muon_step(s["unit"], muon, s["workspace"])
    return {k: s[k] for k in ("master", "exp_avg", "exp_avg_sq", "full_out")}


def _bytes(n):
    return torch.empty(max(1, n), dtype=torch.uint8, device="cuda")


_run_plain = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "ns": _plain_ns, "muon": _plain_muon}
_run_own = {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "ns": _own_ns, "muon": _own_muon}


# ------------------------------------------------------- the 64-bit values


def exact(case, seed):
    if case["op"] in ("ns", "muon") and _ns_flops(_shapes(case["shapes"])) > 6e12:
        return None  # minutes of 64-bit products
    s = prepare(case, seed)
    wide = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point() and v.element_size() > 1}
    return {"norm": _exact_norm, "norm_bwd": _exact_norm_bwd, "ns": _exact_ns, "muon": _exact_muon}[case["op"]](s, wide)


def _exact_norm(s, wide):
    h = wide["x"] + wide["residual"] if s["residual"] is not None else wide["x"]
    size = torch.sqrt((h * h).sum(1) / s["cols"] + s["eps"])
    y = torch.einsum("rc,r,c->rc", h, 1 / size, wide["gain"])
    out = {"rstd": 1 / size}
    if s["residual"] is not None:
        out["h"] = h
    if s["scales"] is not None:
        group = s["group"] or s["cols"]
        which = torch.arange(s["cols"], device="cuda") // group
        scales = torch.zeros(s["rows"], int(which[-1]) + 1, dtype=torch.float64, device="cuda")
        scales.scatter_reduce_(1, which.expand(s["rows"], -1), y.abs(), "amax")
        out["scales"] = torch.clamp(scales / E4M3_MAX, min=TINY)
        y = y / out["scales"][:, which]  # before it is rounded to 8 bits
    out["y"] = y
    return out


def _exact_norm_bwd(s, wide):
    h, dy, r, g = wide["h"], wide["dy"], wide["rstd"], wide["gain"]
    inner = torch.einsum("rc,rc,c->r", dy, h, g)
    dx = torch.einsum("rc,c,r->rc", dy, g, r) - h * (inner * r ** 3 / s["cols"])[:, None]
    if s["dh"] is not None:
        dx = dx + wide["dh"]
    return {"dx": dx, "dgain": torch.einsum("rc,rc,r->c", dy, h, r)}


def _exact_orthogonal(g):
    """Newton-Schulz on the Gram side alone: X_k = Q_k G with Q_k a polynomial of G G^T."""
    wide = g.shape[0] <= g.shape[1]
    x = (g if wide else g.mT).double()
    x = x / (torch.linalg.vector_norm(x) + 1e-7)
    gram = x @ x.mT
    q = torch.eye(x.shape[0], dtype=torch.float64, device=x.device)
    a, b, c = COEFFICIENTS
    for _ in range(5):
        now = q @ gram @ q  # q and gram commute
        step = b * now + c * (now @ now)
        step.diagonal().add_(a)
        q = step @ q
    x = q @ x
    return x if wide else x.mT


def _exact_ns(s, wide):
    return [_exact_orthogonal(g) for g in s["sources"]]


def _exact_muon(s, wide):
    g = wide["grads"].mean(0)
    out = {k: wide[k].clone() for k in ("master", "exp_avg", "exp_avg_sq")}
    at = 0
    for shape in _shapes(s["shapes"]):
        span = torch.arange(at, at + math.prod(shape), device="cuda")
        at += math.prod(shape)
        p, m, v = (out[k][span] for k in ("master", "exp_avg", "exp_avg_sq"))
        if len(shape) == 2:
            m = s["momentum"] * m + g[span]
            u = s["momentum"] * m + g[span] if s["nesterov"] else m
            step = _scale(*shape) * _exact_orthogonal(u.view(shape)).reshape(-1) + s["decay"] * p
        else:
            m = 0.9 * m + (1 - 0.9) * g[span]
            v = 0.95 * v + (1 - 0.95) * g[span] ** 2
            step = m / (1 - 0.9 ** s["adam_step"]) / (torch.sqrt(v / (1 - 0.95 ** s["adam_step"])) + 1e-8)
        out["master"][span], out["exp_avg"][span], out["exp_avg_sq"][span] = p - s["lr"] * step, m, v
    out["full_out"] = out["master"]
    return out
