"""Cases of the feed-forward operators: the gated block, quantisation to 8-bit integers and
products of those.

A gated feed-forward block y = (act(x Wg^T) * (x Wu^T)) Wd^T is trained in bf16 and served in bf16
or in 8-bit integers; dense, or as the networks of an expert layer, each with its run of rows:

  ffn       the block's forward pass, or a training step's forward and backward pass
  quantize  rows to 8-bit integers with a scale each; or, between the block's products, the rows
            act(a) * b of [a | b]
  product   products of such integers with a scale for each row (token) and each channel

Each case is run in a plain form of elementary torch operations or, with `own`, by the calls a
user makes of the package.
"""

import math

import torch

own = False

BLOCK = 128  # the experts' runs of rows start at multiples of this


# ------------------------------------------------------------------------------------- cases


def listed():
    return [
        # one token of a decoding step through the 4096-wide block: latency and weight bandwidth
        dict(name="ffn_one_token", op="ffn", groups=0, rows=1, hidden=4096, inner=14336,
             act="silu", backward=False),
        # one token through eight of 128 experts
        dict(name="ffn_experts_one_token", op="ffn", groups=128, rows=8, hidden=2048, inner=768,
             act="silu", backward=False),
        # a batch of decoding requests
        dict(name="ffn_decode_batch", op="ffn", groups=0, rows=48, hidden=4096, inner=14336,
             act="silu", backward=False),
        # a small training step with odd widths and another activation
        dict(name="ffn_train_odd", op="ffn", groups=0, rows=1000, hidden=1037, inner=515,
             act="gelu", backward=True),
        # a training step of the 4096-wide block
        dict(name="ffn_train_dense", op="ffn", groups=0, rows=8192, hidden=4096, inner=14336,
             act="silu", backward=True),
        # a training step of 128 experts, each token in eight of them
        dict(name="ffn_train_experts", op="ffn", groups=128, rows=65536, hidden=2048, inner=768,
             act="silu", backward=True),
        # one token's inner row on the way to the down projection
        dict(name="quantize_gate_one_token", op="quantize", rows=1, cols=14336, dtype="bf16",
             act="silu"),
        # a prompt's rows before the up projection
        dict(name="quantize_prompt", op="quantize", rows=8192, cols=4096, dtype="bf16", act=""),
        # an odd number of gated rows in fp32
        dict(name="quantize_gate_odd", op="quantize", rows=3001, cols=2053, dtype="f32",
             act="gelu_tanh"),
        # one token's up projection
        dict(name="product_one_token", op="product", groups=0, rows=1, n=14336, k=4096,
             out="bf16"),
        # a prompt's up projection
        dict(name="product_prompt", op="product", groups=0, rows=8192, n=14336, k=4096,
             out="bf16"),
        # the experts' up projections (gate and linear part) for a prompt of an odd length
        dict(name="product_experts", op="product", groups=128, rows=16001, n=1536, k=2048,
             out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["ffn", "ffn", "quantize", "product", "product"])
    if op == "ffn":
        groups = rng.choice([0, 0, 8, 64, 128])
        return dict(op="ffn", groups=groups, rows=_log(rng, 1, 16384),
                    hidden=rng.choice([_log(rng, 16, 2048), 768, 2048]),
                    inner=rng.choice([_log(rng, 16, 2048), 768, 1536]),
                    act=rng.choice(["silu", "gelu", "gelu_tanh"]), backward=rng.random() < 0.6)
    if op == "quantize":
        act = rng.choice(["", "silu", "gelu", "gelu_tanh"])
        return dict(op="quantize", rows=_log(rng, 1, 16384),
                    cols=rng.choice([_log(rng, 1, 16384), 2048, 4096]),
                    dtype=rng.choice(["f32", "bf16"]), act=act)
    return dict(op="product", groups=rng.choice([0, 0, 8, 64, 128]), rows=_log(rng, 1, 16384),
                n=rng.choice([_log(rng, 16, 4096), 768, 1536, 4096]),
                k=rng.choice([_log(rng, 16, 4096), 768, 2048, 4096]),
                out=rng.choice(["f32", "bf16"]))


# ------------------------------------------------------------------------------------ inputs

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _counts(g, groups, rows):
    """How many rows each expert gets: some experts are more popular than others."""
    p = torch.exp(0.5 * _randn(g, groups))
    if rows <= groups:  # one token's experts are distinct
        chosen = p.multinomial(rows, replacement=False, generator=g)
    else:
        chosen = p.multinomial(rows, replacement=True, generator=g)
    return torch.bincount(chosen, minlength=groups)


def _rows(case, g, s):
    """The runs of the experts in `s`; (number of rows, which of them hold a token)."""
    E, R = case["groups"], case["rows"]
    if E == 0:
        s["offsets"] = s["counts"] = None
        s["longest"] = R
        return R, torch.ones(R, 1, dtype=torch.bool, device="cuda")
    counts = _counts(g, E, R)
    size = (counts + BLOCK - 1) // BLOCK * BLOCK
    off = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    off[1:] = size.cumsum(0)
    # rows that always hold the padded runs, whatever their sizes
    total = (R + (BLOCK - 1) * min(E, R)) // BLOCK * BLOCK
    row = torch.arange(total, device="cuda")
    e = (torch.searchsorted(off, row, right=True) - 1).clamp_max(E - 1)
    s["offsets"], s["counts"] = off.to(torch.int32), counts.to(torch.int32)
    s["longest"] = int(size.max())
    return total, (row - off[e] < counts[e])[:, None]


def _codes(x):
    """x in 8-bit integers with a scale for each row, rows padded to 16 bytes."""
    amax = x.abs().amax(-1, keepdim=True).clamp_min(1e-30)
    codes = torch.zeros(*x.shape[:-1], -(-x.shape[-1] // 16) * 16, dtype=torch.int8, device="cuda")
    codes[..., :x.shape[-1]] = torch.round(x * (127.0 / amax)).to(torch.int8)
    return codes[..., :x.shape[-1]], (amax / 127.0)[..., 0].contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op, E = case["op"], case["groups"] if "groups" in case else 0
    stack = (E,) if E else ()
    s = dict(case=dict(case))
    if op == "ffn":
        K, N = case["hidden"], case["inner"]
        total, real = _rows(case, g, s)
        # normalised tokens; weights that keep the activations' size
        s["x"] = torch.where(real, _randn(g, total, K), 0.0).to(torch.bfloat16)
        s["up"] = (_randn(g, *stack, 2 * N, K) * K ** -0.5).to(torch.bfloat16)
        s["down"] = (_randn(g, *stack, K, N) * N ** -0.5).to(torch.bfloat16)
        if case["backward"]:
            s["dy"] = torch.where(real, 0.01 * _randn(g, total, K), 0.0).to(torch.bfloat16)
    elif op == "quantize":
        R, C = case["rows"], case["cols"] * (2 if case["act"] else 1)
        # rows of differing size, a few large entries, one empty row
        x = _randn(g, R, C) * torch.exp(0.5 * _randn(g, R, 1)) * torch.exp(0.5 * _randn(g, 1, C))
        if R > 2:
            x[R // 2] = 0.0
        s["x"] = x.to(_DT[case["dtype"]])
    else:
        K, N = case["k"], case["n"]
        total, real = _rows(case, g, s)
        a = _randn(g, total, K) * torch.exp(0.5 * _randn(g, total, 1))
        s["a"], s["a_scales"] = _codes(torch.where(real, a, 0.0))
        s["b"], s["b_scales"] = _codes(0.02 * _randn(g, *stack, N, K))
    return s


# --------------------------------------------------------------------------------- one pass


def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    import matrix_aware_optimizers_gb300 as mao

    c = s["case"]
    if c["op"] == "ffn":
        kw = dict(act=c["act"], offsets=s["offsets"], counts=s["counts"])
        if not c["backward"]:
            return mao.gated_ffn(s["x"], s["up"], s["down"], **kw)
        y, z = mao.gated_ffn(s["x"], s["up"], s["down"], save=True, **kw)
        dx, dup, ddown = mao.gated_ffn_backward(s["dy"], s["x"], s["up"], s["down"], z, **kw)
        return dict(y=y, dx=dx, dup=dup, ddown=ddown)
    if c["op"] == "quantize":
        return list(mao.int8_quantize(s["x"], gate=c["act"] or None))
    return mao.int8_product(s["a"], s["a_scales"], s["b"], s["b_scales"], offsets=s["offsets"],
                            counts=s["counts"], out_dtype=_DT[c["out"]])


def _plain(s):
    return dict(ffn=_plain_ffn, quantize=_plain_quantize, product=_plain_product)[s["case"]["op"]](s)


def _act(x, name):
    if name == "silu":
        return x / (1.0 + torch.exp(-x))
    if name == "gelu":
        return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))
    return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))


def _act_slope(x, name):
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-x))
        return p * (1.0 + x * (1.0 - p))
    if name == "gelu":
        phi = torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))
        return 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5))) + x * phi
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (x + 0.044715 * x * x * x))
    return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * x * x)


def _split(s, *rows):
    """Rows [R, C] as [groups, longest, C], short runs filled up with zeros."""
    if s["offsets"] is None:
        return [x.float()[None] for x in rows]
    off = s["offsets"].long()
    at = off[:-1, None] + torch.arange(s["longest"], device=off.device)
    inside = (at < off[1:, None])[:, :, None]
    at = torch.where(inside[:, :, 0], at, 0)
    return [torch.where(inside, x.float()[at], 0.0) for x in rows]


def _join(s, y, total):
    """_split's rows in their places again, zeros past the last run."""
    if s["offsets"] is None:
        return y[0]
    off = s["offsets"].long()
    row = torch.arange(total, device=y.device)
    e = torch.searchsorted(off, row, right=True) - 1
    inside = e < len(off) - 1
    e = torch.where(inside, e, 0)
    return torch.where(inside[:, None], y[e, torch.where(inside, row - off[e], 0)], 0.0)


def _stacked(s, w):
    return w.float() if s["offsets"] is not None else w.float()[None]


def _plain_ffn(s):
    c, total = s["case"], len(s["x"])
    up, down = _stacked(s, s["up"]), _stacked(s, s["down"])
    bf16 = torch.bfloat16
    x, = _split(s, s["x"])
    z = torch.bmm(x, up.transpose(1, 2))
    gate, lin = z[:, :, :c["inner"]], z[:, :, c["inner"]:]
    act = _act(gate, c["act"])
    h = act * lin
    y = _join(s, torch.bmm(h, down.transpose(1, 2)), total).to(bf16)
    if not c["backward"]:
        return y
    dy, = _split(s, s["dy"])
    ddown = torch.bmm(dy.transpose(1, 2), h)
    dh = torch.bmm(dy, down)
    dz = torch.cat([dh * lin * _act_slope(gate, c["act"]), dh * act], 2)
    dup = torch.bmm(dz.transpose(1, 2), x)
    dx = _join(s, torch.bmm(dz, up), total)
    if s["offsets"] is None:
        dup, ddown = dup[0], ddown[0]
    return dict(y=y, dx=dx.to(bf16), dup=dup.to(bf16), ddown=ddown.to(bf16))


def _plain_quantize(s):
    c, x = s["case"], s["x"].float()
    if c["act"]:
        x = _act(x[:, :c["cols"]], c["act"]) * x[:, c["cols"]:]
    amax = x.abs().amax(1, keepdim=True)
    # 127 x / amax in 64 bits: nearer to its value than that can be to a border between codes
    q = torch.round(127.0 * x.double() / torch.where(amax > 0, amax, 1.0).double())
    return [q.to(torch.int8), amax[:, 0] / 127.0]


def _plain_product(s):
    c = s["case"]
    a, = _split(s, s["a"])
    y = _join(s, torch.bmm(a, _stacked(s, s["b"]).transpose(1, 2)), len(s["a"]))
    y = y * s["a_scales"][:, None]
    if s["offsets"] is None:
        return (y * s["b_scales"]).to(_DT[c["out"]])
    row = torch.arange(len(y), device=y.device)
    e = (torch.searchsorted(s["offsets"].long(), row, right=True) - 1).clamp_max(c["groups"] - 1)
    return (y * s["b_scales"][e]).to(_DT[c["out"]])


# ----------------------------------------------------------------------------------- 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return dict(ffn=_exact_ffn, quantize=_exact_quantize, product=_exact_product)[case["op"]](s)


def _exact_gate(a, b, name):
    f = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
         "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[name]
    return f(a) * b


def _runs(s, total):
    if s["offsets"] is None:
        return [(0, total)]
    off = s["offsets"].tolist()
    return list(zip(off[:-1], off[1:]))


def _exact_ffn(s):
    c, total = s["case"], len(s["x"])
    if 6.0 * total * c["hidden"] * c["inner"] * (3 if c["backward"] else 1) > 2.5e12:
        return None
    one = s["offsets"] is None
    up = (s["up"][None] if one else s["up"])
    down = (s["down"][None] if one else s["down"])
    y = torch.zeros(total, c["hidden"], dtype=torch.float64, device="cuda")
    out = dict(y=y)
    if c["backward"]:
        out["dx"] = torch.zeros_like(y)
        out["dup"] = torch.zeros(up.shape, dtype=torch.float64, device="cuda")
        out["ddown"] = torch.zeros(down.shape, dtype=torch.float64, device="cuda")
    for e, (lo, hi) in enumerate(_runs(s, total)):
        if hi == lo:
            continue
        leaves = [t.double().requires_grad_(c["backward"]) for t in (s["x"][lo:hi], up[e], down[e])]
        x, wu, wd = leaves
        g, u = (x @ wu.T).split(c["inner"], 1)
        r = _exact_gate(g, u, c["act"]) @ wd.T
        y[lo:hi] = r.detach()
        if c["backward"]:
            r.backward(s["dy"][lo:hi].double())
            out["dx"][lo:hi], out["dup"][e], out["ddown"][e] = (t.grad for t in leaves)
    if not c["backward"]:
        return y
    if one:
        out["dup"], out["ddown"] = out["dup"][0], out["ddown"][0]
    return out


def _exact_quantize(s):
    c, x = s["case"], s["x"].double()
    if c["act"]:
        x = _exact_gate(x[:, :c["cols"]], x[:, c["cols"]:], c["act"])
    # the codes are whole numbers, those of gated rows by the values' rounding to 32 bits
    return [None, x.abs().amax(1) / 127.0]


def _exact_product(s):
    c, total = s["case"], len(s["a"])
    if 2.0 * total * c["n"] * c["k"] > 1.2e12:
        return None
    b = s["b"] if s["offsets"] is not None else s["b"][None]
    bs = s["b_scales"] if s["offsets"] is not None else s["b_scales"][None]
    y = torch.zeros(total, c["n"], dtype=torch.float64, device="cuda")
    for e, (lo, hi) in enumerate(_runs(s, total)):
        a = s["a"][lo:hi].double() * s["a_scales"][lo:hi, None].double()
        y[lo:hi] = a @ (b[e].double() * bs[e][:, None].double()).T
    return y


# -------------------------------------------------------------------------------------- work


def work(case):
    op, R = case["op"], case["rows"]
    E = case["groups"] if "groups" in case else 0
    used = min(E, R) if E else 1  # experts whose weights are read
    if op == "ffn":
        K, N = case["hidden"], case["inner"]
        weights = 3 * K * N
        b, f = 2 * (used * weights + 2 * R * K), 2 * R * weights
        if case["backward"]:
            # dY and X in, dX out, the weights again, their gradients out
            b, f = b + 2 * (3 * R * K + (used + max(E, 1)) * weights), 3 * f
        return dict(bytes=b, flops=f)
    if op == "quantize":
        C, es = case["cols"], 4 if case["dtype"] == "f32" else 2
        return dict(bytes=R * C * (es * (2 if case["act"] else 1) + 1) + 4 * R,
                    flops=R * C * (13 if case["act"] else 3))
    N, K = case["n"], case["k"]
    es = 4 if case["out"] == "f32" else 2
    return dict(bytes=R * K + used * N * K + R * N * es + 4 * (R + used * N), flops=2 * R * N * K)
