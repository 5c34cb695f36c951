"""The cases that the experts' products and the gradients' norm are measured on: what a training step does between the
dispatch of tokens to experts and their combination, backwards, and with all gradients before the weights are changed.

  gated       rows sorted by expert through the expert's gate and up projections, act(gate) * up, forward; optionally the
              two projections are kept for the backward pass
  gated_bwd   its gradient towards the projections, the rows and both weights
  linear      rows sorted by expert through one projection of their expert (the block's way down)
  linear_bwd  its gradient towards the rows and the weights
  clip        the global norm over many gradient tensors and, with max_norm, the gradients scaled down to it
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZE = {"bf16": 2, "f16": 2, "f32": 4}
EPS = 1e-6
DEV = "cuda:0"
ACTS = ("silu", "gelu", "gelu_tanh")


# ------------------------------------------------------------------------------------------------ cases
def _product(name, op, tokens, k, experts, hidden, inner, dtype, act="silu", align=1, save=False):
    """experts 0: one matrix for all tokens (a dense block)."""
    return {"name": name, "op": op, "tokens": tokens, "k": k, "experts": experts, "hidden": hidden, "inner": inner,
            "dtype": dtype, "act": act, "align": align, "save": save}


def _clip(name, layers, hidden, inner, dtype, max_norm, kind="l2"):
    """The gradients of `layers` layers of `hidden` and `inner` channels; max_norm 0: the norm alone."""
    return {"name": name, "op": "clip", "layers": layers, "hidden": hidden, "inner": inner, "dtype": dtype,
            "max_norm": max_norm, "kind": kind}


def listed():
    return [
        # serving: one token, eight of 64 experts; the weights of eight experts are read for one row each
        _product("gated_one_token", "gated", 1, 8, 64, 2048, 1024, "bf16"),
        # training, forward: a batch to 32 experts, segments padded to a tile's rows, both projections kept
        _product("gated_train", "gated", 8192, 4, 32, 4096, 2048, "bf16", align=128, save=True),
        # a dense block in 32 bits at sizes that nothing divides
        _product("gated_ragged_f32", "gated", 777, 1, 0, 1025, 1371, "f32", act="gelu"),
        # training, backward: half of that batch
        _product("gated_bwd_train", "gated_bwd", 4096, 4, 32, 4096, 2048, "bf16", align=128),
        # a small batch in fp16, odd widths, segments that start anywhere
        _product("gated_bwd_ragged_f16", "gated_bwd", 201, 2, 6, 1190, 530, "f16", act="gelu_tanh"),
        # serving: a decode batch of 48 sequences, one to a few rows for each of 128 experts
        _product("linear_decode", "linear", 48, 4, 128, 1024, 4096, "bf16"),
        # a prompt batch's way down, 64 experts of eight each
        _product("linear_prompt", "linear", 16384, 8, 64, 1024, 2048, "bf16", align=16),
        # training, backward: the way down of a batch to 32 experts
        _product("linear_bwd_train", "linear_bwd", 8192, 4, 32, 2048, 4096, "bf16", align=128),
        # a micro-batch in 32 bits, odd widths
        _product("linear_bwd_ragged_f32", "linear_bwd", 333, 3, 10, 1003, 770, "f32"),
        # the gradients of one small layer: the calls' latency
        _clip("clip_small", 1, 256, 512, "bf16", 0.05),
        # the gradients of a dense model in bf16, its norms' weights in fp32: scaled down
        _clip("clip_large_mixed", 8, 4096, 8192, "mixed", 1.0),
        # the norm alone, in 32 bits, of tensors of odd sizes
        _clip("norm_ragged_f32", 6, 1003, 2050, "f32", 0.0),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width():
        w = spread(64, 4096)
        return -(-w // 64) * 64 if rng.random() < 0.6 else w

    op = rng.choice(["gated", "gated", "gated_bwd", "linear", "linear_bwd", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "clip":
        hidden, inner, dtype = width(), spread(64, 8192), rng.choice([dtype, "mixed"])
        # no more bytes than the largest listed case has
        most = 8 * (4 * 4096 + 3 * 8192) * 4096 * 2 // ((4 * hidden + 3 * inner) * hidden * (4 if dtype == "f32" else 2))
        return {"op": op, "layers": spread(1, max(1, min(40, most))), "hidden": hidden, "inner": inner, "dtype": dtype,
                "max_norm": rng.choice([0.0, spread(1, 100) / 100]), "kind": rng.choice(["l2", "l2", "max"])}
    hidden, inner = width(), width()
    experts = rng.choice([0, 8, 16, 60, 64, 128])
    # the weights of all experts stay below those of the largest listed case
    each = hidden * inner * SIZE[dtype] * (2 if op.startswith("gated") else 1)
    while experts * each > 128 * 1024 * 4096 * 2:
        experts //= 2
    k = rng.randint(1, min(8, experts)) if experts else 1
    products = {"gated": 2, "gated_bwd": 4, "linear": 1, "linear_bwd": 2}[op]
    most = 2 * 8192 * 4 * 4096 * 2048 // (products * k * hidden * inner * (4 if dtype == "f32" else 1))
    return {"op": op, "tokens": spread(1, max(1, min(8192, most))), "k": k, "experts": experts, "hidden": hidden,
            "inner": inner, "dtype": dtype, "act": rng.choice(ACTS), "align": rng.choice([1, 1, 16, 128]),
            "save": op == "gated" and rng.random() < 0.5}


def _widths(c):
    """(what a row holds, what its products hold): `linear` goes from hidden to inner channels as `gated` does."""
    return c["hidden"], c["inner"]


def _shapes(c):
    """The gradient tensors of a model: four square projections, three of the feed-forward block, two norms a layer."""
    h, i = c["hidden"], c["inner"]
    return [((h, h), False)] * 4 * c["layers"] + [((i, h), False)] * 3 * c["layers"] + [((h,), True)] * 2 * c["layers"]


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _matrices(g, n, out, inside, dt):
    w = torch.empty(n, out, inside, dtype=dt, device=DEV)
    for e in range(n):
        w[e] = _randn(g, out, inside) / math.sqrt(inside)
    return w


def _rows(g, where, rows, width, dt, scale=1.0):
    """Rows of different size with a few channels that stand out; what lies between and behind the segments is zero."""
    x = torch.zeros(rows, width, dtype=dt, device=DEV)
    loud = torch.where(torch.rand(width, generator=g, device=DEV) < 0.01, 4.0, 1.0)
    for at in range(0, rows, 16384):
        n = min(16384, rows - at)
        v = _randn(g, n, width) * (0.5 + torch.rand(n, 1, generator=g, device=DEV)) * loud * scale
        x[at:at + n] = torch.where(where[at:at + n, None], v, 0.0).to(dt)
    return x


def _flat(grads, dtype=None):
    """A flat buffer for the tensors of each type, every tensor at a multiple of 16 bytes, and the tensors' places in it."""
    flat, places, ends = {}, [], {}
    for t in grads:
        lo = ends.get(t.dtype, 0)
        places.append((t.dtype, lo, t.shape))
        ends[t.dtype] = lo + -(-t.numel() * t.element_size() // 16) * 16 // t.element_size()
    for dt, end in ends.items():
        flat[str(dt)] = torch.zeros(end, dtype=dtype or dt, device=DEV)
    return flat, [flat[str(dt)][lo:lo + shape.numel()].view(shape) for dt, lo, shape in places]


def prepare(case, seed):
    g, c = _gen(seed), case
    s = {"case": c}
    if c["op"] == "clip":
        s["grads"] = []
        for shape, norm in _shapes(c):
            dt = DTYPES["f32" if norm else "bf16"] if c["dtype"] == "mixed" else DTYPES[c["dtype"]]
            s["grads"].append((_randn(g, *shape) * (0.01 * torch.rand(1, generator=g, device=DEV))).to(dt))
        # the scaled gradients go to one flat buffer per type, as a bucketed all-reduce keeps them
        s["flat"], s["outs"] = _flat(s["grads"]) if c["max_norm"] else (None, None)
        s["norm"] = torch.empty(1, device=DEV)
        if own:
            import all_reduce_reduction_ring_amd as ar
            # the table of the gradients' addresses, which a program builds once
            s["plan"] = ar.ar_grad_plan(s["grads"], s["outs"])
            s["workspace"] = torch.empty(ar.ar_grad_norm_workspace_size(s["plan"].shape[0]), dtype=torch.uint8, device=DEV)
        return s
    dt, n = DTYPES[c["dtype"]], max(c["experts"], 1)
    inside, wide = _widths(c)
    if c["experts"]:
        logits = _randn(g, c["tokens"], n) + 1.5 * _randn(g, 1, n)  # some experts are asked far more often
        ids = logits.topk(c["k"], dim=1)[1]
        counts = torch.bincount(ids.reshape(-1), minlength=n).tolist()
    else:
        counts = [c["tokens"]]
    slots, align = c["tokens"] * c["k"], c["align"] if c["experts"] else 1
    starts = [0]
    for m in counts:
        starts.append(starts[-1] + -(-m // align) * align)
    rows = slots + min(n, slots) * (align - 1)  # the rows that a program sets aside for any choices
    s["rows"], s["segments"] = rows, [(e, starts[e], starts[e] + m) for e, m in enumerate(counts) if m]
    i32 = torch.int32
    s["offsets"] = torch.tensor(starts, dtype=i32, device=DEV) if c["experts"] else None
    s["counts"] = torch.tensor(counts, dtype=i32, device=DEV) if c["experts"] else None
    where = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for _, lo, hi in s["segments"]:
        where[lo:hi] = True
    s["xs"] = _rows(g, where, rows, inside, dt)
    names = ("w_gate", "w_up") if c["op"].startswith("gated") else ("w",)
    for name in names:
        w = _matrices(g, n, wide, inside, dt)
        s[name] = w if c["experts"] else w[0]
    new = lambda width: torch.zeros(rows, width, dtype=dt, device=DEV)
    if c["op"] in ("gated", "linear"):
        s["out"] = new(wide)
        s["gate"], s["up"] = (new(wide), new(wide)) if c["save"] else (None, None)
        return s
    s["dout"] = _rows(g, where, rows, wide, dt, 0.05)
    s["dxs"] = new(inside)
    if c["op"] == "gated_bwd":
        s["gate"], s["up"] = _rows(g, where, rows, wide, dt), _rows(g, where, rows, wide, dt)
        s["dgate"], s["dup"] = new(wide), new(wide)
    for name in names:
        s["d" + name] = torch.empty_like(s[name])
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _act(x, act):
    """The activation and its derivative."""
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-x))
        return x * p, p * (1.0 + x * (1.0 - p))
    if act == "gelu":
        p = 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5)))
        return x * p, p + x * torch.exp(-0.5 * x * x) / math.sqrt(2.0 * math.pi)
    a = math.sqrt(2.0 / math.pi)
    t = torch.tanh(a * (x + 0.044715 * x * x * x))
    return 0.5 * x * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * a * (1.0 + 3.0 * 0.044715 * x * x)


def _of(w, e):
    return (w[e] if w.dim() == 3 else w).float()


def _plain_gated(s):
    c, dt = s["case"], s["xs"].dtype
    out = {"out": torch.zeros_like(s["out"])}
    if c["save"]:
        out["gate"], out["up"] = torch.zeros_like(s["out"]), torch.zeros_like(s["out"])
    for e, lo, hi in s["segments"]:
        x = s["xs"][lo:hi].float()
        gate, up = x @ _of(s["w_gate"], e).t(), x @ _of(s["w_up"], e).t()
        out["out"][lo:hi] = (_act(gate, c["act"])[0] * up).to(dt)
        if c["save"]:
            out["gate"][lo:hi], out["up"][lo:hi] = gate.to(dt), up.to(dt)
    return out


def _plain_gated_bwd(s):
    c, dt = s["case"], s["xs"].dtype
    out = {k: torch.zeros_like(s[k]) for k in ("dgate", "dup", "dxs", "dw_gate", "dw_up")}
    for e, lo, hi in s["segments"]:
        x, dout, up = s["xs"][lo:hi].float(), s["dout"][lo:hi].float(), s["up"][lo:hi].float()
        value, slope = _act(s["gate"][lo:hi].float(), c["act"])
        dgate, dup = dout * up * slope, dout * value
        out["dgate"][lo:hi], out["dup"][lo:hi] = dgate.to(dt), dup.to(dt)
        out["dxs"][lo:hi] = (dgate @ _of(s["w_gate"], e) + dup @ _of(s["w_up"], e)).to(dt)
        for name, d in (("dw_gate", dgate), ("dw_up", dup)):
            w = out[name][e] if c["experts"] else out[name]
            w.copy_((d.t() @ x).to(dt))
    return out


def _plain_linear(s):
    out = torch.zeros_like(s["out"])
    for e, lo, hi in s["segments"]:
        out[lo:hi] = (s["xs"][lo:hi].float() @ _of(s["w"], e).t()).to(out.dtype)
    return {"out": out}


def _plain_linear_bwd(s):
    dt = s["xs"].dtype
    dxs, dw = torch.zeros_like(s["xs"]), torch.zeros_like(s["w"])
    for e, lo, hi in s["segments"]:
        dout = s["dout"][lo:hi].float()
        dxs[lo:hi] = (dout @ _of(s["w"], e)).to(dt)
        (dw[e] if s["case"]["experts"] else dw).copy_((dout.t() @ s["xs"][lo:hi].float()).to(dt))
    return {"dxs": dxs, "dw": dw}


def _plain_clip(s):
    c = s["case"]
    if c["kind"] == "max":
        norm = torch.stack([t.abs().max().float() for t in s["grads"]]).max().view(1)
    else:  # squares of small gradients add up over a billion elements: 64 bits between the tensors
        norm = torch.stack([t.float().square().sum().double() for t in s["grads"]]).sum().sqrt().float().view(1)
    if not c["max_norm"]:
        return {"norm": norm}
    coef = (c["max_norm"] / (norm + EPS)).clamp(max=1.0)
    for t, out in zip(s["grads"], s["outs"]):
        out.copy_(t.float() * coef)
    return {"norm": norm, "outs": s["flat"]}


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    s, c = state, state["case"]
    if not own:
        return {"gated": _plain_gated, "gated_bwd": _plain_gated_bwd, "linear": _plain_linear,
                "linear_bwd": _plain_linear_bwd, "clip": _plain_clip}[c["op"]](s)
    import all_reduce_reduction_ring_amd as ar
    if c["op"] == "clip":
        kind = ar.AR_NORM_MAX if c["kind"] == "max" else ar.AR_NORM_L2
        if not c["max_norm"]:
            ar.ar_grad_norm(s["plan"], s["norm"], kind=kind, workspace=s["workspace"])
            return {"norm": s["norm"]}
        ar.ar_grad_clip(s["plan"], c["max_norm"], s["norm"], kind=kind, eps=EPS, workspace=s["workspace"])
        return {"norm": s["norm"], "outs": s["flat"]}
    seg = {"offsets": s["offsets"], "counts": s["counts"]}
    act = {"silu": ar.AR_ACT_SILU, "gelu": ar.AR_ACT_GELU, "gelu_tanh": ar.AR_ACT_GELU_TANH}[c["act"]]
    if c["op"] == "gated":
        ar.ar_expert_gated(s["xs"], s["w_gate"], s["w_up"], s["out"], gate=s["gate"], up=s["up"], act=act, **seg)
        out = {"out": s["out"]}
        if c["save"]:
            out["gate"], out["up"] = s["gate"], s["up"]
        return out
    if c["op"] == "gated_bwd":
        ar.ar_expert_gated_bwd(s["dout"], s["gate"], s["up"], s["xs"], s["w_gate"], s["w_up"], s["dgate"], s["dup"],
                               dxs=s["dxs"], dw_gate=s["dw_gate"], dw_up=s["dw_up"], act=act, **seg)
        return {k: s[k] for k in ("dgate", "dup", "dxs", "dw_gate", "dw_up")}
    if c["op"] == "linear":
        ar.ar_expert_linear(s["xs"], s["w"], s["out"], **seg)
        return {"out": s["out"]}
    ar.ar_expert_linear_bwd(s["dout"], s["xs"], s["w"], dxs=s["dxs"], dw=s["dw"], **seg)
    return {"dxs": s["dxs"], "dw": s["dw"]}


# ------------------------------------------------------------------------------------------------ what it takes
def work(case):
    c = case
    if c["op"] == "clip":
        elems = sum(math.prod(shape) for shape, _ in _shapes(c))
        nbytes = sum(math.prod(shape) * (SIZE["f32" if norm else "bf16"] if c["dtype"] == "mixed" else SIZE[c["dtype"]])
                     for shape, norm in _shapes(c))
        return {"bytes": nbytes * (2 if c["max_norm"] else 1), "flops": elems * (3 if c["max_norm"] else 2)}
    es, slots = SIZE[c["dtype"]], c["tokens"] * c["k"]
    inside, wide = _widths(c)
    n = max(c["experts"], 1)
    # the experts that some token has chosen, taking the choices as even: a token's are different ones
    used = n * (1.0 - (1.0 - c["k"] / n) ** c["tokens"]) if c["experts"] else 1
    w = int(used * inside * wide) * es
    x, y, product = slots * inside * es, slots * wide * es, 2 * slots * inside * wide
    if c["op"] == "gated":
        return {"bytes": x + 2 * w + y * (3 if c["save"] else 1), "flops": 2 * product}
    if c["op"] == "linear":
        return {"bytes": x + w + y, "flops": product}
    all_w = n * inside * wide * es  # the gradient of an expert without rows is written too
    if c["op"] == "gated_bwd":
        return {"bytes": 2 * x + 5 * y + 2 * w + 2 * all_w, "flops": 4 * product}
    return {"bytes": 2 * x + y + w + all_w, "flops": 2 * product}


# ------------------------------------------------------------------------------------------------ in 64 bits
def _act64(x, act):
    if act == "silu":
        return x * torch.sigmoid(x)
    if act == "gelu":
        return x * torch.special.ndtr(x)
    return x * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x.pow(3)))


def exact(case, seed):
    c, s, f64 = case, prepare(case, seed), torch.float64
    if c["op"] == "clip":
        if c["kind"] == "max":
            norm = max(float(t.abs().max()) for t in s["grads"])
        else:
            norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(t, dtype=f64)) ** 2 for t in s["grads"]))
        out = {"norm": torch.tensor([norm], dtype=f64, device=DEV)}
        if c["max_norm"]:
            out["outs"], places = _flat(s["grads"], f64)
            for t, place in zip(s["grads"], places):
                torch.mul(t.to(f64), min(1.0, c["max_norm"] / (norm + EPS)), out=place)
        return out
    wide = lambda t: torch.zeros(t.shape, dtype=f64, device=DEV)
    one = lambda w, e: (w[e] if c["experts"] else w)
    names = {"gated": ["out"] + ["gate", "up"] * c["save"], "gated_bwd": ["dgate", "dup", "dxs", "dw_gate", "dw_up"],
             "linear": ["out"], "linear_bwd": ["dxs", "dw"]}[c["op"]]
    out = {k: wide(s[k]) for k in names}
    for e, lo, hi in s["segments"]:
        x = s["xs"][lo:hi].to(f64)
        if c["op"] == "linear":
            out["out"][lo:hi] = torch.mm(x, one(s["w"], e).to(f64).t())
        elif c["op"] == "gated":
            gate, up = torch.mm(x, one(s["w_gate"], e).to(f64).t()), torch.mm(x, one(s["w_up"], e).to(f64).t())
            out["out"][lo:hi] = _act64(gate, c["act"]) * up
            if c["save"]:
                out["gate"][lo:hi], out["up"][lo:hi] = gate, up
        else:
            dout = s["dout"][lo:hi].to(f64)
            if c["op"] == "linear_bwd":
                parts = [(dout, "w")]
            else:
                with torch.enable_grad():  # the gradients of the block's own definition
                    gate = s["gate"][lo:hi].to(f64).requires_grad_()
                    up = s["up"][lo:hi].to(f64).requires_grad_()
                    dgate, dup = torch.autograd.grad(_act64(gate, c["act"]) * up, (gate, up), dout)
                out["dgate"][lo:hi], out["dup"][lo:hi] = dgate, dup
                parts = [(dgate, "w_gate"), (dup, "w_up")]
            for d, name in parts:
                out["dxs"][lo:hi] += torch.mm(d, one(s[name], e).to(f64))
                one(out["d" + name], e).copy_(torch.mm(d.t().contiguous(), x))
    return out
