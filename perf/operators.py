"""Cases of the expert-layer operators: routing, 8-bit quantisation, 8-bit products, combination.

An expert layer sends each token to a few of many experts, multiplies it by their matrices and
adds the results up. Its operators, in the order of a training step:

  route     scores of the experts for each token, the choice of the best (masks, a bias for
            balance, groups of experts), the plan of where each token's copies go, and the
            gradient of the logits
  quantize  tensors to 8-bit floating point (e4m3) with a power-of-two scale for each block of
            128 entries of a row, of a column, or 128 x 128, with the gather of the dispatch
  product   products of such tensors with 32-bit sums, dense or over the experts' groups of
            rows: "nt" (forward), "nn" (gradient of the input), "tn" (gradient of the weights)
  combine   the weighted sum of a token's expert outputs, and its gradients

Each case is run in a plain form of elementary torch operations or, with `own`, by the calls a
user makes of the package.
"""

import math

import torch

own = False

BLOCK = 128


# ------------------------------------------------------------------------------------- cases


def listed():
    return [
        # one token of a decoding step: latency of the choice and its plan
        dict(name="route_one_token", op="route", tokens=1, experts=128, top_k=8, score="softmax",
             dtype="f32", bias=False, groups=1, keep=1, renorm=True, masked=False, backward=False),
        # a training step with balance bias and groups of experts, padding tokens masked
        dict(name="route_train_groups", op="route", tokens=16384, experts=256, top_k=8,
             score="sigmoid", dtype="f32", bias=True, groups=8, keep=4, renorm=True, masked=True,
             backward=True),
        # the dispatch of a training step: gathered rows, in both block directions
        dict(name="quantize_dispatch", op="quantize", batch=1, rows=8192, cols=2048, dtype="bf16",
             blocks="both", gather=8),
        # all experts' up projections after an optimizer step
        dict(name="quantize_experts", op="quantize", batch=128, rows=1536, cols=2048,
             dtype="bf16", blocks="tile", gather=0),
        # a few odd rows in fp32
        dict(name="quantize_odd_rows", op="quantize", batch=1, rows=1000, cols=1037, dtype="f32",
             blocks="row", gather=0),
        # a dense projection of the 4096-wide layers
        dict(name="product_dense_nt", op="product", form="nt", groups=0, rows=8192, n=14336,
             k=4096, out="bf16"),
        # experts' up projection in a training step
        dict(name="product_experts_nt", op="product", form="nt", groups=128, rows=65536, n=1536,
             k=2048, out="bf16"),
        # the same for one token of a decoding step: the weights of eight experts
        dict(name="product_one_token_nt", op="product", form="nt", groups=128, rows=8, n=1536,
             k=2048, out="bf16"),
        # gradient of the down projection's input, an odd number of tokens
        dict(name="product_experts_nn", op="product", form="nn", groups=128, rows=60007, n=2048,
             k=768, out="bf16"),
        # gradient of the up projections' weights, kept in fp32
        dict(name="product_experts_tn", op="product", form="tn", groups=128, rows=65536, n=1536,
             k=2048, out="f32"),
        # one token's eight expert outputs
        dict(name="combine_one_token", op="combine", tokens=1, top_k=8, width=2048, dtype="bf16",
             experts=128, backward=False),
        # a training step, with the gradients of outputs and weights
        dict(name="combine_train", op="combine", tokens=8192, top_k=8, width=2048, dtype="bf16",
             experts=128, backward=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "quantize", "product", "product", "combine"])
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        experts = groups * rng.choice([8, 16, 20, 32]) if groups > 1 else rng.choice([8, 60, 64, 128, 200, 256])
        keep = rng.randint(max(1, groups // 2), groups)
        return dict(op="route", tokens=_log(rng, 1, 16384), experts=experts,
                    top_k=rng.randint(1, min(8, experts * keep // groups)),
                    score=rng.choice(["softmax", "sigmoid"]), dtype=rng.choice(["f32", "bf16"]),
                    bias=rng.random() < 0.5, groups=groups, keep=keep, renorm=rng.random() < 0.7,
                    masked=rng.random() < 0.5, backward=rng.random() < 0.6)
    if op == "quantize":
        blocks = rng.choice(["row", "col", "tile", "both"])
        gather = rng.choice([0, 0, 1, 4, 8]) if blocks in ("row", "both") else 0
        batch = _log(rng, 1, 64) if gather == 0 else 1
        return dict(op="quantize", batch=batch, rows=_log(rng, 1, 32768 // max(batch, gather)),
                    cols=rng.choice([_log(rng, 16, 4096), 768, 1536, 2048, 4096]),
                    dtype=rng.choice(["f32", "bf16"]), blocks=blocks, gather=gather)
    if op == "product":
        form = rng.choice(["nt", "nn", "tn"])
        groups = rng.choice([0, 8, 32, 128])
        return dict(op="product", form=form, groups=groups, rows=_log(rng, 1, 32768),
                    n=rng.choice([_log(rng, 16, 2048), 768, 1536, 2048]),
                    k=rng.choice([_log(rng, 16, 2048), 768, 1536, 2048]),
                    out=rng.choice(["f32", "bf16"]))
    return dict(op="combine", tokens=_log(rng, 1, 4096), top_k=rng.randint(1, 8),
                width=rng.choice([_log(rng, 16, 4096), 768, 2048]),
                dtype=rng.choice(["f32", "bf16"]), experts=rng.choice([8, 64, 128]),
                backward=rng.random() < 0.6)


# ------------------------------------------------------------------------------------ inputs

_DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _keys(logits, case, bias):
    """Selection keys in 64 bits, masked experts at -inf."""
    x = logits.double()
    if bias is None and case["groups"] == 1:
        return x
    s = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.softmax(x, 1).nan_to_num(0.0)
    s = s if bias is None else s + bias.double()
    return torch.where(x == -math.inf, -math.inf, s)


def _near(order):
    """Where neighbours of descending keys differ, but by next to nothing."""
    a, b = order[:, :-1], order[:, 1:]
    gap = (a - b).abs()
    return (gap > 0) & (gap < 1e-5 * (a.abs() + b.abs()) + 1e-7)


def _undecided(logits, case, bias):
    """Rows whose choice rests on the last bits of two scores: no two programs, and no two
    precisions, need to agree on those."""
    key = _keys(logits, case, bias)
    T, G, E, k = len(key), case["groups"], case["experts"], case["top_k"]
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    if bias is None and G == 1:
        return bad  # the logits themselves decide
    if G > 1:
        two = key.view(T, G, E // G).topk(min(2, E // G), 2).values
        score = torch.where(two == -math.inf, 0.0, two).sum(2)
        score = torch.where(two[:, :, 0] == -math.inf, -math.inf, score)
        order, at = score.sort(dim=1, descending=True, stable=True)
        bad |= _near(order)[:, case["keep"] - 1:case["keep"]].any(1)
        kept = torch.zeros_like(score, dtype=torch.bool).scatter_(1, at[:, :case["keep"]], True)
        key = key.masked_fill(~kept.repeat_interleave(E // G, 1), -math.inf)
    return bad | _near(key.sort(1, descending=True).values[:, :k + 1]).any(1)


def _logits(case, g):
    T, E = case["tokens"], case["experts"]
    bias = 0.05 * _randn(g, E) if case["bias"] else None
    # experts differ in popularity; logits of a linear layer over normalised tokens
    popular = 0.5 * _randn(g, E)

    def rows(n):
        x = (popular + 1.5 * _randn(g, n, E)).to(_DT[case["dtype"]])
        if case["masked"]:
            x[torch.rand(n, E, generator=g, device="cuda") < 0.1] = -math.inf  # full experts
            x[torch.rand(n, generator=g, device="cuda") < 0.02] = -math.inf    # padding tokens
        return x

    x = rows(T)
    for _ in range(64):  # draw rows whose choice is not decided at 32 bits again
        bad = _undecided(x, case, bias).nonzero().flatten()
        if not len(bad):
            break
        x[bad] = rows(len(bad))
    return x, bias


def _counts(g, groups, rows):
    """How many rows each expert gets: some experts are more popular than others."""
    p = torch.exp(0.5 * _randn(g, groups))
    if rows <= groups:  # one token's experts are distinct
        chosen = p.multinomial(rows, replacement=False, generator=g)
    else:
        chosen = p.multinomial(rows, replacement=True, generator=g)
    return torch.bincount(chosen, minlength=groups)


def _capacity(rows, groups):
    """Rows that always hold the padded groups, whatever their sizes: what a program allocates
    that does not wait for the routing's result."""
    return (rows + (BLOCK - 1) * min(groups, rows)) // BLOCK * BLOCK


def _padded(counts):
    """Row offsets of the groups, each group padded to whole blocks."""
    size = (counts + BLOCK - 1) // BLOCK * BLOCK
    off = torch.zeros(len(counts) + 1, dtype=torch.int64, device="cuda")
    off[1:] = size.cumsum(0)
    return off


def _rows_of_groups(counts, capacity):
    """Offsets of the padded groups and which of the rows hold something."""
    off = _padded(counts)
    row = torch.arange(capacity, device="cuda")
    e = torch.searchsorted(off, row, right=True) - 1
    e = e.clamp_max(len(counts) - 1)
    return off, row - off[e] < counts[e]


def _codes(x, blocks):
    """x in e4m3 with exponent bytes, rows padded to 16 bytes: ready-made operands."""
    B, R, C = x.shape
    br, bc = {"row": (1, BLOCK), "col": (BLOCK, 1), "tile": (BLOCK, BLOCK)}[blocks]
    pr, pc = -R % br, -C % bc
    y = torch.nn.functional.pad(x, (0, pc, 0, pr)).view(B, (R + pr) // br, br, (C + pc) // bc, bc)
    amax = y.abs().amax((2, 4), keepdim=True).clamp_min(2.0 ** -100)
    e = torch.ceil(torch.log2(amax / 448.0))
    e = torch.where(amax <= 448.0 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(amax > 448.0 * torch.exp2(e), e + 1, e)
    y = (y * torch.exp2(-e)).view(B, R + pr, C + pc)[:, :R, :C]
    codes = torch.zeros(B, R, -(-C // 16) * 16, dtype=torch.float8_e4m3fn, device="cuda")
    codes.view(torch.uint8)[:, :, :C] = y.to(torch.float8_e4m3fn).view(torch.uint8)
    return codes[:, :, :C], (e + 127).to(torch.uint8)[:, :, 0, :, 0].contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    s = dict(case=dict(case))
    if op == "route":
        s["logits"], s["bias"] = _logits(case, g)
        s["dweights"] = _randn(g, case["tokens"], case["top_k"]) if case["backward"] else None
    elif op == "quantize":
        B, R, C = case["batch"], case["rows"], case["cols"]
        # rows and columns of differing size, a few large entries, one empty row
        x = _randn(g, B, R, C) * torch.exp(_randn(g, B, R, 1)) * torch.exp(0.5 * _randn(g, B, 1, C))
        x[:, R // 2] = 0.0
        s["x"] = x.to(_DT[case["dtype"]])
        s["src"] = None
        if case["gather"]:
            # the copies of each token in the order of the experts, with padding rows between
            copies = R * case["gather"]
            total = _capacity(copies, 128)
            _, real = _rows_of_groups(_counts(g, 128, copies), total)
            src = torch.randint(0, R, (total,), generator=g, device="cuda")
            s["src"] = torch.where(real, src, -1).to(torch.int32)
    elif op == "product":
        E, R, N, K = case["groups"], case["rows"], case["n"], case["k"]
        if E:
            total = _capacity(R, E)
            off, real = _rows_of_groups(_counts(g, E, R), total)
            real = real[:, None]
            s["offsets"], s["longest"] = off.to(torch.int32), int((off[1:] - off[:-1]).max())
        else:
            total, real, s["offsets"], s["longest"] = R, True, None, R
        form = case["form"]
        a = _randn(g, total, K if form == "nt" else N) * torch.exp(0.5 * _randn(g, total, 1))
        a = torch.where(real, a, 0.0) if E else a
        s["a"], s["a_scales"] = _codes(a[None], "col" if form == "tn" else "row")
        if form == "tn":
            b = _randn(g, total, K) * torch.exp(0.5 * _randn(g, total, 1))
            b = torch.where(real, b, 0.0) if E else b
            s["b"], s["b_scales"] = _codes(b[None], "col")
            s["b"], s["b_scales"] = s["b"][0], s["b_scales"][0]
        else:
            s["b"], s["b_scales"] = _codes(0.02 * _randn(g, max(E, 1), N, K), "tile")
        s["a"], s["a_scales"] = s["a"][0], s["a_scales"][0]
    else:
        T, k, H, E = case["tokens"], case["top_k"], case["width"], case["experts"]
        # distinct experts for each token, and their copies' places among the padded groups
        ids = (_randn(g, T, E) + 0.5 * _randn(g, E)).topk(k, 1).indices
        off = _padded(torch.bincount(ids.flatten(), minlength=E))
        order = ids.flatten().argsort(stable=True)
        first = torch.searchsorted(ids.flatten()[order], torch.arange(E, device="cuda"))
        rank = torch.arange(T * k, device="cuda") - first[ids.flatten()[order]]
        row_of = torch.empty(T * k, dtype=torch.int64, device="cuda")
        row_of[order] = off[ids.flatten()[order]] + rank
        s["row_of"] = row_of.view(T, k).to(torch.int32)
        rows = _capacity(T * k, E)
        s["z"] = _randn(g, rows, H).to(_DT[case["dtype"]])
        w = torch.rand(T, k, generator=g, device="cuda") + 0.1
        s["weights"] = w / w.sum(1, keepdim=True)
        s["dy"] = _randn(g, T, H).to(_DT[case["dtype"]]) if case["backward"] else None
        src = torch.full((rows,), -1, dtype=torch.int64, device="cuda")
        src[row_of] = torch.arange(T * k, device="cuda")
        s["slot_of"] = src.to(torch.int32)
    return s


# --------------------------------------------------------------------------------- one pass


def run(state):
    return (_own if own else _plain)(state)


def _own(s):
    import matrix_aware_optimizers_gb300 as mao

    c = s["case"]
    if c["op"] == "route":
        opts = dict(score=c["score"], renorm=c["renorm"])
        w, ids = mao.expert_route(s["logits"], c["top_k"], bias=s["bias"], groups=c["groups"],
                                  keep_groups=c["keep"], group_score="top2", **opts)
        plan = mao.expert_plan(ids, c["experts"])
        out = dict(weights=w, ids=ids, counts=plan.counts, offsets=plan.offsets,
                   row_of=plan.row_of, slot_of=plan.slot_of)
        if c["backward"]:
            out["dlogits"] = mao.expert_route_backward(s["logits"], ids, s["dweights"], **opts)
        return out
    if c["op"] == "quantize":
        return list(mao.fp8_quantize(s["x"], c["blocks"], rows=s["src"]))
    if c["op"] == "product":
        return mao.fp8_product(s["a"], s["a_scales"], s["b"], s["b_scales"], c["form"],
                               offsets=s["offsets"], out_dtype=_DT[c["out"]])
    y = mao.expert_combine(s["z"], s["row_of"], s["weights"])
    if not c["backward"]:
        return y
    dz, dw = mao.expert_combine_backward(s["dy"], s["z"], s["row_of"], s["slot_of"], s["weights"])
    return dict(y=y, dz=dz, dw=dw)


def _plain(s):
    return dict(route=_plain_route, quantize=_plain_quantize, product=_plain_product,
                combine=_plain_combine)[s["case"]["op"]](s)


def _best(key, k):
    """Positions of the k largest keys of each row, ties to the lower position."""
    return torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]


def _plain_route(s):
    c, x = s["case"], s["logits"].float()
    T, E, G, k = c["tokens"], c["experts"], c["groups"], c["top_k"]
    open_ = x > -math.inf
    if c["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-x))
    else:
        top = x.amax(1, keepdim=True)
        p = torch.exp(x - torch.where(top > -math.inf, top, 0.0))
        p = p / p.sum(1, keepdim=True).clamp_min(1e-37)
    key = x if s["bias"] is None and G == 1 else p if s["bias"] is None else p + s["bias"]
    key = torch.where(open_, key, -math.inf)
    if G > 1:
        sort = torch.sort(key.view(T, G, E // G), 2, descending=True).values[:, :, :2]
        score = torch.where(sort > -math.inf, sort, 0.0).sum(2)
        score = torch.where(sort[:, :, 0] > -math.inf, score, -math.inf)
        kept = torch.zeros(T, G, dtype=torch.bool, device=x.device)
        kept.scatter_(1, _best(score, c["keep"]), True)
        key = torch.where(kept[:, :, None].expand(T, G, E // G).reshape(T, E), key, -math.inf)
    ids = _best(key, k)
    taken = key.gather(1, ids) > -math.inf
    chosen = torch.where(taken, p.gather(1, ids), 0.0)
    total = chosen.sum(1, keepdim=True) + 1e-20
    w = chosen / total if c["renorm"] else chosen
    ids = torch.where(taken, ids, -1)

    # the plan: where each copy goes among groups of whole blocks, in the order of the tokens
    flat = torch.where(ids >= 0, ids, E).flatten()
    order = torch.sort(flat, stable=True).indices
    counts = torch.zeros(E + 1, dtype=torch.int64, device=x.device)
    counts.index_add_(0, flat, torch.ones_like(flat))
    size = (counts[:E] + BLOCK - 1) // BLOCK * BLOCK
    off = torch.cat([size.new_zeros(1), size.cumsum(0)])
    start = torch.cat([counts.new_zeros(1), counts.cumsum(0)])[:-1]
    sorted_ids = flat[order]
    rank = torch.arange(T * k, device=x.device) - start[sorted_ids]
    place = torch.where(sorted_ids < E, off[sorted_ids] + rank, -1)
    row_of = torch.empty(T * k, dtype=torch.int64, device=x.device)
    row_of[order] = place
    rows = _capacity(T * k, E)
    slot_of = torch.full((rows + 1,), -1, dtype=torch.int64, device=x.device)
    slot_of[torch.where(place >= 0, place, rows)] = torch.where(place >= 0, order, -1)
    i32 = torch.int32
    out = dict(weights=w, ids=ids.to(i32), counts=counts[:E].to(i32), offsets=off.to(i32),
               row_of=row_of.view(T, k).to(i32), slot_of=slot_of[:rows].to(i32))
    if c["backward"]:
        d = s["dweights"]
        if c["renorm"]:
            d = torch.where(taken, (d - (d * w).sum(1, keepdim=True)) / total, 0.0)
        else:
            d = torch.where(taken, d, 0.0)
        ds = torch.zeros(T, E + 1, device=x.device)
        ds = ds.scatter_(1, torch.where(taken, ids, E), d)[:, :E]
        if c["score"] == "sigmoid":
            dx = ds * p * (1.0 - p)
        else:
            dx = p * (ds - (ds * p).sum(1, keepdim=True))
        out["dlogits"] = dx.to(s["logits"].dtype)
    return out


def _plain_blocks(x, br, bc):
    """x [B, R, C] in e4m3 with the exponent bytes of br x bc blocks."""
    B, R, C = x.shape
    pr, pc = -R % br, -C % bc
    y = torch.nn.functional.pad(x, (0, pc, 0, pr)).view(B, (R + pr) // br, br, (C + pc) // bc, bc)
    amax = y.abs().amax((2, 4), keepdim=True)
    m, q = torch.frexp(amax)  # amax = m 2^q with m in [0.5, 1): 448 2^e = 0.875 2^(e + 9)
    e = torch.where(m <= 0.875, q - 9, q - 8).clamp(min=-127)
    e = torch.where(amax > 0, e, -127)
    y = torch.ldexp(y, -e).view(B, R + pr, C + pc)[:, :R, :C]
    return y.to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)[:, :, 0, :, 0]


def _plain_quantize(s):
    c, x = s["case"], s["x"].float()
    if s["src"] is not None:
        src = s["src"].long()
        x = torch.where(src[None, :, None] >= 0, x[:, src.clamp_min(0)], 0.0)
    row = _plain_blocks(x, 1, BLOCK) if c["blocks"] in ("row", "both") else ()
    col = _plain_blocks(x, BLOCK, 1) if c["blocks"] in ("col", "both") else ()
    tile = _plain_blocks(x, BLOCK, BLOCK) if c["blocks"] == "tile" else ()
    return list(row + col + tile)


def _values(codes, scales, br, bc):
    """The 32-bit values of codes [B, R, C] with one exponent byte per br x bc block."""
    B, R, C = codes.shape
    f = torch.exp2(scales.float() - 127.0)
    f = f[:, :, None, :, None].expand(B, f.shape[1], br, f.shape[2], bc)
    return codes.float() * f.reshape(B, f.shape[1] * br, -1)[:, :R, :C]


def _by_group(x, off, longest):
    """Rows [R, C] as [groups, longest, C], short groups filled up with zeros."""
    at = off[:-1, None] + torch.arange(longest, device=x.device)
    inside = at < off[1:, None]
    return torch.where(inside[:, :, None], x[torch.where(inside, at, 0)], 0.0)


def _plain_product(s):
    c = s["case"]
    form, dt = c["form"], _DT[c["out"]]
    if form == "tn":
        a = _values(s["a"][None], s["a_scales"][None], BLOCK, 1)[0]
        b = _values(s["b"][None], s["b_scales"][None], BLOCK, 1)[0]
        if s["offsets"] is None:
            return (a.T @ b)[None].to(dt)
        off = s["offsets"].long()
        a, b = _by_group(a, off, s["longest"]), _by_group(b, off, s["longest"])
        return torch.bmm(a.transpose(1, 2), b).to(dt)
    a = _values(s["a"][None], s["a_scales"][None], 1, BLOCK)[0]
    b = _values(s["b"], s["b_scales"], BLOCK, BLOCK)
    b = b.transpose(1, 2) if form == "nt" else b
    if s["offsets"] is None:
        return (a @ b[0]).to(dt)
    off = s["offsets"].long()
    y = torch.bmm(_by_group(a, off, s["longest"]), b)
    row = torch.arange(len(a), device=a.device)
    e = torch.searchsorted(off, row, right=True) - 1
    inside = e < len(off) - 1
    e = torch.where(inside, e, 0)
    return torch.where(inside[:, None], y[e, torch.where(inside, row - off[e], 0)], 0.0).to(dt)


def _plain_combine(s):
    c, at, w = s["case"], s["row_of"].long(), s["weights"]
    z = s["z"][at].float()
    y = (w[:, :, None] * z).sum(1).to(s["z"].dtype)
    if not c["backward"]:
        return y
    dy = s["dy"].float()
    dw = (z * dy[:, None, :]).sum(2)
    dz = torch.zeros(s["z"].shape, device=z.device)
    dz[at] = w[:, :, None] * dy[:, None, :]
    return dict(y=y, dz=dz.to(s["z"].dtype), dw=dw)


# ----------------------------------------------------------------------------------- 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return dict(route=_exact_route, quantize=_exact_quantize, product=_exact_product,
                combine=_exact_combine)[case["op"]](s)


def _exact_route(s):
    c, x = s["case"], s["logits"].double()
    T, E, k = c["tokens"], c["experts"], c["top_k"]
    key = _keys(s["logits"], c, s["bias"])
    if c["groups"] > 1:
        by = key.view(T, c["groups"], -1)
        first = by.amax(2)
        if by.shape[2] > 1:
            second = by.sort(2).values[:, :, -2]
            score = first + torch.where(second == -math.inf, 0.0, second)
        else:
            score = first
        best = (-score).argsort(dim=1, stable=True)[:, :c["keep"]]
        keep = torch.zeros_like(score, dtype=torch.bool).scatter_(1, best, True)
        key = key.masked_fill(~keep.repeat_interleave(E // c["groups"], 1), -math.inf)
    ids = (-key).argsort(dim=1, stable=True)[:, :k]
    on = key.gather(1, ids) != -math.inf
    leaf = x.clone().requires_grad_(True)
    dead = (x == -math.inf).all(1, keepdim=True)
    p = torch.sigmoid(leaf) if c["score"] == "sigmoid" else torch.softmax(leaf.masked_fill(dead, 0.0), 1)
    w = p.gather(1, ids) * on
    if c["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    out = dict(weights=w.detach(), ids=None, counts=None, offsets=None, row_of=None, slot_of=None)
    if c["backward"]:
        w.backward(s["dweights"].double())
        out["dlogits"] = leaf.grad.nan_to_num(0.0)
    return out


def _exact_quantize(s):
    c, x = s["case"], s["x"].double()
    if s["src"] is not None:
        src = s["src"].long()
        x = x[:, src.clamp_min(0)] * (src >= 0)[None, :, None]
    out = []
    for name in ("row", "col") if c["blocks"] == "both" else (c["blocks"],):
        br, bc = {"row": (1, BLOCK), "col": (BLOCK, 1), "tile": (BLOCK, BLOCK)}[name]
        B, R, C = x.shape
        y = torch.zeros(B, -(-R // br) * br, -(-C // bc) * bc, dtype=torch.float64, device="cuda")
        y[:, :R, :C] = x
        y = y.unflatten(1, (-1, br)).unflatten(3, (-1, bc))
        amax = y.abs().amax((2, 4), keepdim=True)
        e = torch.full_like(amax, -127.0)
        for step in (128, 64, 32, 16, 8, 4, 2, 1):  # the smallest exponent that holds amax
            e = torch.where(448.0 * torch.exp2(e + step - 1) < amax, e + step, e)
        v = y / torch.exp2(e)
        # e4m3: three bits after the leading one, steps of 2^-9 below 2^-6, ties to even
        ulp = torch.exp2(torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -6))) - 3)
        v = torch.round(v / ulp) * ulp
        out += [v.flatten(3, 4).flatten(1, 2)[:, :R, :C], None]
    return out


def _exact_product(s):
    c = s["case"]
    off = [0, len(s["a"])] if s["offsets"] is None else s["offsets"].tolist()

    def whole(codes, scales, br, bc):
        f = torch.exp2(scales.double() - 127).repeat_interleave(br, 0).repeat_interleave(bc, 1)
        return codes.double() * f[:codes.shape[0], :codes.shape[1]]

    if 2.0 * len(s["a"]) * c["n"] * c["k"] > 1.2e12:
        return None
    form, out = c["form"], []
    for g, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        if form == "tn":
            sl = slice(lo // BLOCK, -(-hi // BLOCK))
            out.append(whole(s["a"][lo:hi], s["a_scales"][sl], BLOCK, 1).T
                       @ whole(s["b"][lo:hi], s["b_scales"][sl], BLOCK, 1))
        elif hi > lo:
            a = whole(s["a"][lo:hi], s["a_scales"][lo:hi], 1, BLOCK)
            b = whole(s["b"][g], s["b_scales"][g], BLOCK, BLOCK)
            out.append(a @ (b.T if form == "nt" else b))
    if form == "tn":
        return torch.stack(out)
    y = torch.cat(out)  # rows past the last group are zero
    return torch.nn.functional.pad(y, (0, 0, 0, len(s["a"]) - len(y)))


def _exact_combine(s):
    c, at, w = s["case"], s["row_of"].long(), s["weights"].double()
    T, k = at.shape
    y = torch.zeros(T, c["width"], dtype=torch.float64, device="cuda")
    dz = torch.zeros(len(s["z"]), c["width"], dtype=torch.float64, device="cuda")
    dw = torch.zeros(T, k, dtype=torch.float64, device="cuda")
    for j in range(k):
        z = s["z"][at[:, j]].double()
        y += w[:, j:j + 1] * z
        if c["backward"]:
            dy = s["dy"].double()
            dw[:, j] = torch.einsum("th,th->t", z, dy)
            dz[at[:, j]] = w[:, j:j + 1] * dy
    return dict(y=y, dz=dz, dw=dw) if c["backward"] else y


# -------------------------------------------------------------------------------------- work


def work(case):
    op = case["op"]
    if op == "route":
        T, E, k = case["tokens"], case["experts"], case["top_k"]
        es = 4 if case["dtype"] == "f32" else 2
        # logits in; weights and ids out; the plan: ids in, places and slots out
        b = T * E * es + T * k * (8 + 4 + 4 + 4) + 8 * E
        f = 10 * T * E
        if case["backward"]:
            b += 2 * T * E * es + 8 * T * k
            f += 8 * T * E
        return dict(bytes=b, flops=f)
    if op == "quantize":
        B, R, C = case["batch"], case["rows"], case["cols"]
        es = 4 if case["dtype"] == "f32" else 2
        out = B * R * C * max(1, case["gather"])
        two = 2 if case["blocks"] == "both" else 1
        return dict(bytes=B * R * C * es + out * two + out * two // BLOCK, flops=3 * out * two)
    if op == "product":
        E, R, N, K = case["groups"], case["rows"], case["n"], case["k"]
        es = 4 if case["out"] == "f32" else 2
        used = min(max(E, 1), R) if E else 1  # experts whose weights are read
        a = R * (K if case["form"] == "nt" else N)
        if case["form"] == "tn":
            b = a + R * K + max(E, 1) * N * K * es
        else:
            b = a + used * N * K + R * (N if case["form"] == "nt" else K) * es
        return dict(bytes=b, flops=2 * R * N * K)
    T, k, H = case["tokens"], case["top_k"], case["width"]
    es = 4 if case["dtype"] == "f32" else 2
    b, f = (T * k + T) * H * es + 8 * T * k, 2 * T * k * H
    if case["backward"]:
        b, f = b + (2 * T * k + T) * H * es + 12 * T * k, 3 * f
    return dict(bytes=b, flops=f)
