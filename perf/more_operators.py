"""What the operators of an expert layer's training are measured on: routing with its balance loss, the exchange of
tokens with their experts' rows, and activations that are kept in 8 bits for the backward pass.

`route`     the k largest logits of each token, their weights, every expert's count and rows, and the balance loss; with
            `grad` also the backward pass, as a training step runs both
`act`       an activation with the codes of its result (the next product's operand) and, with `keep`, of its argument
            (the checkpoint)
`dact`      the backward pass from the checkpoint: codes of the argument's gradient along the rows and transposed, and
            the transposed codes of the activation, computed again
`recode`    transposed codes (one factor per 128 tokens) of a checkpoint that was kept along the rows
`exchange`  tokens quantised into their experts' rows ("dispatch"), the weighted sum of what comes back ("combine"),
            and that sum with its gradients ("train")

Codes are FP8 with one fp32 factor per 128 values.  `own` is false: plain torch in fp32; true: the framework's entry
points.
"""
import torch

own = False

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FP8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
HP = {"bf16": torch.bfloat16, "fp32": torch.float32}
CODE = {"e4m3": 0, "e5m2": 1}
ACT = {"gelu": 0, "silu": 1, "geglu": 2, "swiglu": 3}
TINY = 2.0 ** -100  # a smaller block maximum counts as this one (its reciprocal stays finite)


def listed():
    return [
        # decoding: one new token chooses among the experts (latency)
        dict(name="route 1 of 64", op="route", tokens=1, experts=64, k=6, x="bf16", padded=0, closed=0, normalize=True, grad=False),
        # a training step with few large experts
        dict(name="route 4096 of 8", op="route", tokens=4096, experts=8, k=2, x="fp32", padded=0, closed=0, normalize=True, grad=True),
        # a training step with many small experts, padded sequences, weights as the softmax gives them
        dict(name="route 32768 of 256", op="route", tokens=32768, experts=256, k=8, x="bf16", padded=1000, closed=0, normalize=False, grad=True),
        # serving: 128 routed rows of 24 experts between the two products, nothing kept
        dict(name="act 128x1408 swiglu", op="act", rows=128, cols=1408, act="swiglu", x="bf16", q="e4m3", groups=24, behind=0, keep=False),
        # training: a gated MLP at ffn 11008, argument kept in 8 bits
        dict(name="act 8192x11008 swiglu", op="act", rows=8192, cols=11008, act="swiglu", x="bf16", q="e4m3", groups=0, behind=0, keep=True),
        # the backward pass of the same, with the bias gradient
        dict(name="dact 8192x11008 swiglu", op="dact", rows=8192, cols=11008, act="swiglu", x="bf16", q="e4m3", groups=0, behind=0, dbias=True),
        # small experts with few tokens each, plain GELU, fp32 gradients into E5M2
        dict(name="dact 2999x1408 gelu", op="dact", rows=2999, cols=1408, act="gelu", x="fp32", q="e5m2", groups=24, behind=100, dbias=False),
        # an expert layer's input: 16384 tokens kept once, each in two experts' weight gradients
        dict(name="recode 32768x4096", op="recode", source=16384, rows=32768, cols=4096, q="e4m3", to="e4m3", groups=16, behind=64, index=True),
        # one linear layer's input, kept along the rows only
        dict(name="recode 3001x2048", op="recode", source=3001, rows=3001, cols=2048, q="e4m3", to="e4m3", groups=0, behind=0, index=False),
        # training: tokens into the rows of 16 experts, and a copy in their own order as the checkpoint
        dict(name="dispatch 16384x4096", op="exchange", what="dispatch", tokens=16384, experts=16, k=2, cols=4096, x="bf16", q="e4m3", padded=32, keep=True),
        # decoding: a small batch comes back from its experts
        dict(name="combine 37x4096", op="exchange", what="combine", tokens=37, experts=64, k=6, cols=4096, x="bf16", q="e4m3", padded=0, keep=False),
        # training: the weighted sum and its gradients
        dict(name="combine 16384x4096 train", op="exchange", what="train", tokens=16384, experts=16, k=2, cols=4096, x="bf16", q="e4m3", padded=32, keep=False),
    ]


def _log(rng, lo, hi, step=1):
    """A size between lo and hi, spread over its logarithm, a multiple of step."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random() / step)) * step))


def draw(rng):
    op = rng.choice(["route", "route", "act", "dact", "dact", "recode", "exchange", "exchange"])
    if op == "route":
        experts, tokens = _log(rng, 2, 256), _log(rng, 1, 16384)
        return dict(op=op, tokens=tokens, experts=experts, k=rng.randint(1, min(8, experts)), x=rng.choice(["bf16", "fp32"]),
                    padded=rng.choice([0, rng.randint(0, tokens // 2)]), closed=rng.choice([0, rng.randint(0, experts // 2)]),
                    normalize=rng.random() < 0.5, grad=rng.random() < 0.7)
    if op in ("act", "dact"):
        groups, rows = rng.choice([0, rng.randint(1, 64)]), _log(rng, 1, 8192)
        c = dict(op=op, rows=rows, cols=_log(rng, 128, 8192, 16), act=rng.choice(["gelu", "silu", "geglu", "swiglu"]),
                 x=rng.choice(["bf16", "fp32"]), q=rng.choice(["e4m3", "e5m2"]) if op == "dact" else "e4m3", groups=groups,
                 behind=rng.randint(0, min(70, rows // 2)) if groups else 0)
        c["keep" if op == "act" else "dbias"] = rng.random() < 0.5 and (op == "act" or not groups)
        return c
    if op == "recode":
        groups, index = rng.choice([0, rng.randint(1, 64)]), rng.random() < 0.5
        rows = _log(rng, 1, 16384)
        return dict(op=op, source=_log(rng, 1, 16384) if index else rows, rows=rows, cols=_log(rng, 128, 8192, 16),
                    q=rng.choice(["e4m3", "e5m2"]), to=rng.choice(["e4m3", "e5m2"]), groups=groups,
                    behind=rng.randint(0, min(70, rows // 2)) if groups else 0, index=index)
    tokens, experts = _log(rng, 1, 4096), _log(rng, 2, 128)
    return dict(op=op, what=rng.choice(["dispatch", "combine", "train"]), tokens=tokens, experts=experts, k=rng.randint(1, min(6, experts)),
                cols=_log(rng, 128, 3328, 16), x=rng.choice(["bf16", "fp32"]), q=rng.choice(["e4m3", "e5m2"]),
                padded=rng.choice([0, rng.randint(0, tokens // 2)]), keep=rng.random() < 0.5)


def _ceil(a, b):
    return (a + b - 1) // b


def _capacity(rows, groups):
    """Columns of the transposed codes: every group padded to a multiple of 128, at most this many in all."""
    return (rows + 127 * min(groups, rows)) // 128 * 128


def _gated(case):
    return case["act"] in ("geglu", "swiglu")


# ------------------------------------------------------------------------------------------------ plain forms
def _scales(amax, fmt):
    """(scale, stored factor) of blocks with these maxima: scale = fp8_max / amax, factor = 1 / scale; 1 where a
    block holds nothing."""
    one = torch.ones_like(amax)
    scale = torch.where(amax > 0, (one * FP8_MAX[fmt]) / amax.clamp(min=TINY), one)  # tensor by tensor: a true division
    return scale, one / scale


def _codes(x, scale, fmt):
    return (x * scale).clamp(-FP8_MAX[fmt], FP8_MAX[fmt]).to(F8[fmt])


def _pad128(x, dim):
    n = x.shape[dim]
    p = _ceil(n, 128) * 128 - n
    return torch.nn.functional.pad(x, (0, p) if dim == x.dim() - 1 else (0, 0, 0, p)) if p else x


def _quantize_rows(x, fmt):
    """Row-wise: codes [R, C] and factors [C / 128, R]."""
    r, c = x.shape
    xb = _pad128(x.float(), 1).view(r, -1, 128)
    scale, inv = _scales(xb.abs().amax(2), fmt)
    return _codes(xb, scale[:, :, None], fmt).view(r, -1)[:, :c], inv.t().contiguous()


def _quantize_cols(x, fmt):
    """Along the rows, x's rows being a multiple of 128: transposed codes [C, R] and factors [R / 128, C]."""
    r, c = x.shape
    xb = x.float().view(-1, 128, c)
    scale, inv = _scales(xb.abs().amax(1), fmt)
    return _codes(xb, scale[:, None, :], fmt).view(r, c).view(torch.uint8).t().contiguous().view(F8[fmt]), inv


def _slots(off, rows, groups):
    """For each column of the padded, transposed codes: its row (`rows` where it has none); whether a group has it."""
    n = off[1:] - off[:-1]
    pad = torch.cumsum((n + 127) // 128 * 128, 0)
    at = torch.arange(_capacity(rows, groups), device=off.device)
    g = torch.searchsorted(pad, at, right=True)
    inside = g < groups
    g = g.clamp(max=groups - 1)
    k = at - (pad - (n + 127) // 128 * 128)[g]
    return torch.where(inside & (k < n[g]), off[:-1][g] + k, torch.full_like(at, rows)), inside


def _transposed(x, fmt, off, groups):
    """Transposed codes and factors of x's groups; zeros behind the last."""
    if off is None:
        return _quantize_cols(_pad128(x, 0), fmt)
    src, inside = _slots(off.long(), x.shape[0], groups)
    q, s = _quantize_cols(torch.cat([x, torch.zeros_like(x[:1])])[src], fmt)
    return q, torch.where(inside[::128][:, None], s, 0.0)


def _rowwise(x, fmt, off):
    """Row-wise codes and factors; zeros outside the groups."""
    q, s = _quantize_rows(x, fmt)
    if off is None:
        return q, s
    at = torch.arange(x.shape[0], device=x.device)
    used = (at >= off[0]) & (at < off[-1])
    return torch.where(used[:, None], q.view(torch.uint8), 0).view(F8[fmt]), torch.where(used[None, :], s, 0.0)


def _values(q, fmt, s):
    """The numbers that codes q [R, K] with factors s [K / 128, R] stand for."""
    return q.view(F8[fmt]).float() * s.t().repeat_interleave(128, 1)[:, :q.shape[1]]


def _act(a, kind):
    """act(a) and its derivative."""
    if kind in ("gelu", "geglu"):
        phi = 0.5 * (1.0 + torch.erf(a * 0.7071067811865476))
        return a * phi, phi + a * torch.exp(-0.5 * a * a) * 0.3989422804014327
    s = 1.0 / (1.0 + torch.exp(-a))
    return a * s, s * (1.0 + a * (1.0 - s))


def _route(case, logits, valid):
    """(chosen experts, which of them there are, softmax over all experts of the counted tokens, weights)."""
    l = logits.float()
    if valid is not None:
        l = torch.where(valid[:, None], l, -torch.inf)
    top, expert = torch.sort(l, dim=1, descending=True, stable=True)
    has = top[:, :case["k"]] > -torch.inf
    e = torch.where(has[:, :1], torch.exp(l - torch.where(has[:, :1], top[:, :1], 0.0)), 0.0)
    p = e / torch.where(has[:, :1], e.sum(1, keepdim=True), 1.0)
    expert = expert[:, :case["k"]]
    w = torch.where(has, p.gather(1, expert), 0.0)
    if case["normalize"]:
        w = w / torch.where(has[:, :1], w.sum(1, keepdim=True), 1.0)
    return expert, has, p, w


# ------------------------------------------------------------------------------------------------ inputs
def _activation(rows, cols, g, dtype, spread=0.7):
    """Normal values with a spread of channel sizes, as activations have."""
    ch = torch.exp(torch.randn(cols, device="cuda", generator=g) * spread)
    return (torch.randn((rows, cols), device="cuda", generator=g) * ch).to(dtype)


def _offsets(rows, behind, groups, seed):
    """Uneven groups over the rows but the last `behind`, in no order of size; some are empty where rows are few."""
    rows = max(0, rows - behind)
    w = [1.0 / (i + 1) ** 0.7 for i in range(groups)]
    n = [int(rows * v / sum(w)) for v in w]
    n[0] += rows - sum(n)
    order = torch.randperm(groups, generator=torch.Generator().manual_seed(seed))
    off = torch.zeros(groups + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(torch.tensor(n, dtype=torch.int32)[order], 0)
    return off.cuda()


def _tokens_valid(tokens, padded):
    """Sequences end in padding: `padded` tokens are none, up to 64 at the end of each sequence."""
    seqs = _ceil(padded, 64)
    valid = torch.ones(tokens, dtype=torch.bool)
    for i in range(seqs):
        end = tokens // seqs * (i + 1)
        valid[end - padded // seqs - (i < padded % seqs):end] = False
    return valid.cuda()


def _positions(case, g):
    """Where a routing of unevenly wanted experts puts each token's copies: [tokens, k] int32, -1 for padding."""
    t, e, k = case["tokens"], case["experts"], case["k"]
    want = torch.randn((t, e), device="cuda", generator=g) + torch.randn(e, device="cuda", generator=g)
    expert = torch.topk(want, k, 1).indices
    if case["padded"]:
        expert = torch.where(_tokens_valid(t, case["padded"])[:, None], expert, e)
    order = torch.sort(expert.reshape(-1), stable=True).indices
    pos = torch.empty_like(order)
    pos[order] = torch.arange(t * k, device="cuda")
    return torch.where(expert < e, pos.view(t, k), -1).int().contiguous()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st, op = dict(case=case), case["op"]
    u8, f32, i32 = dict(dtype=torch.uint8, device="cuda"), dict(device="cuda"), dict(dtype=torch.int32, device="cuda")
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["k"]
        bias = torch.randn(e, device="cuda", generator=g) * 0.5
        logits = torch.randn((t, e), device="cuda", generator=g) * 1.5 + bias
        if case["closed"]:  # experts that take no tokens now
            logits[:, torch.randperm(e, device="cuda", generator=g)[:case["closed"]]] = -torch.inf
        st["logits"] = logits.to(HP[case["x"]])
        st["valid"] = _tokens_valid(t, case["padded"]) if case["padded"] else None
        st["expert"], st["weight"] = torch.empty((t, k), **i32), torch.empty((t, k), **f32)
        st["position"], st["token"] = torch.empty((t, k), **i32), torch.full((t * k,), -1, **i32)
        st["offsets"], st["counts"] = torch.empty(e + 1, **i32), torch.empty(e, **i32)
        st["slope"], st["loss"] = torch.empty(e, **f32), torch.empty(1, **f32)
        st["dweight"] = torch.randn((t, k), device="cuda", generator=g) * 1e-2
        st["dloss"] = torch.full((1,), 1e-2 * (1 + seed % 7), **f32)
        st["dlogits"] = torch.empty_like(st["logits"])
        st["ws"] = torch.empty(8 * 160 * (e + 1) + 64, **u8)
    elif op == "act":
        r, c = case["rows"], case["cols"]
        wide = 2 * c if _gated(case) else c
        st["h"] = _activation(r, wide, g, HP[case["x"]])
        st["g_q"], st["g_s"] = torch.zeros((r, c), **u8), torch.zeros((_ceil(c, 128), r), **f32)
        keep = case["keep"]
        st["h_q"], st["h_s"] = (torch.zeros((r, wide), **u8), torch.zeros((_ceil(wide, 128), r), **f32)) if keep else (None, None)
        st["off"] = _offsets(r, case["behind"], case["groups"], seed) if case["groups"] else None
    elif op == "dact":
        r, c = case["rows"], case["cols"]
        wide, cap = 2 * c if _gated(case) else c, _capacity(r, max(1, case["groups"]))
        q, st["h_s"] = _quantize_rows(_activation(r, wide, g, HP["bf16"]), "e4m3")
        st["h_q"] = q.contiguous().view(torch.uint8)
        st["dg"] = (_activation(r, c, g, HP["fp32"], 0.5) * 1e-3).to(HP[case["x"]])
        st["off"] = _offsets(r, case["behind"], case["groups"], seed) if case["groups"] else None
        st["dh_q"], st["dh_s"] = torch.zeros((r, wide), **u8), torch.zeros((_ceil(wide, 128), r), **f32)
        st["dh_qt"], st["dh_st"] = torch.zeros((wide, cap), **u8), torch.zeros((cap // 128, wide), **f32)
        st["g_qt"], st["g_st"] = torch.zeros((c, cap), **u8), torch.zeros((cap // 128, c), **f32)
        st["db"] = torch.empty(wide, **f32) if case["dbias"] else None
        st["ws"] = torch.empty(_ceil(r, 128) * wide * 4, **u8) if case["dbias"] else None
    elif op == "recode":
        r, c, cap = case["rows"], case["cols"], _capacity(case["rows"], max(1, case["groups"]))
        q, st["s"] = _quantize_rows(_activation(case["source"], c, g, HP["bf16"]), case["q"])
        st["q"] = q.contiguous().view(torch.uint8)
        st["off"] = _offsets(r, case["behind"], case["groups"], seed) if case["groups"] else None
        st["index"] = torch.randint(0, case["source"], (r,), device="cuda", generator=g).int() if case["index"] else None
        st["col_q"], st["col_s"] = torch.zeros((c, cap), **u8), torch.zeros((cap // 128, c), **f32)
    else:
        t, k, c = case["tokens"], case["k"], case["cols"]
        st["position"] = _positions(case, g)
        if case["what"] == "dispatch":
            st["x"] = _activation(t, c, g, HP[case["x"]])
            st["row_q"], st["row_s"] = torch.zeros((t * k, c), **u8), torch.zeros((_ceil(c, 128), t * k), **f32)
            keep = case["keep"]
            st["q"], st["s"] = (torch.zeros((t, c), **u8), torch.zeros((_ceil(c, 128), t), **f32)) if keep else (None, None)
        else:
            w = torch.rand((t, k), device="cuda", generator=g) + 0.05
            st["weight"] = w / w.sum(1, keepdim=True)
            st["y"] = _activation(t * k, c, g, HP[case["x"]])
            st["out"] = torch.empty((t, c), dtype=HP[case["x"]], device="cuda")
            if case["what"] == "train":
                st["dout"] = (_activation(t, c, g, HP["fp32"], 0.5) * 1e-3).to(HP[case["x"]])
                st["dy"], st["dweight"] = torch.zeros_like(st["y"]), torch.empty((t, k), **f32)
    torch.cuda.synchronize()
    return st


# ------------------------------------------------------------------------------------------------ one pass
def run(st):
    if own:
        return _own(st)
    case = st["case"]
    op = case["op"]
    if op == "route":
        return _plain_route(case, st)
    if op == "act":
        h, c, fmt = st["h"].float(), case["cols"], case["q"]
        y = _act(h[:, :c], case["act"])[0]
        out = dict(zip(("g_q", "g_s"), _rowwise(y * h[:, c:] if _gated(case) else y, fmt, st["off"])))
        if case["keep"]:
            out["h_q"], out["h_s"] = _rowwise(h, fmt, st["off"])
        return out
    if op == "dact":
        h, c, dg, off = _values(st["h_q"], "e4m3", st["h_s"]), case["cols"], st["dg"].float(), st["off"]
        y, d = _act(h[:, :c], case["act"])
        u = h[:, c:] if _gated(case) else None
        dh = dg * d if u is None else torch.cat([dg * u * d, dg * y], 1)
        out = dict(zip(("dh_q", "dh_s"), _rowwise(dh, case["q"], off)))
        out["dh_qt"], out["dh_st"] = _transposed(dh, case["q"], off, case["groups"])
        out["g_qt"], out["g_st"] = _transposed(y if u is None else y * u, "e4m3", off, case["groups"])
        if case["dbias"]:
            out["dbias"] = dh.sum(0)
        return out
    if op == "recode":
        x = _values(st["q"], case["q"], st["s"])
        if st["index"] is not None:
            x = x[st["index"]]
        q, s = _transposed(x, case["to"], st["off"], case["groups"])
        return dict(col_q=q, col_s=s)
    pos, k = st["position"].long(), case["k"]
    used = pos >= 0
    if case["what"] == "dispatch":
        q, s = _quantize_rows(st["x"], case["q"])
        rows = q.shape[0] * k
        at = torch.where(used, pos, rows).view(-1)
        row_q = torch.zeros((rows + 1, case["cols"]), dtype=torch.uint8, device="cuda")
        row_q[at] = q.view(torch.uint8).repeat_interleave(k, 0)
        row_s = torch.zeros((s.shape[0], rows + 1), device="cuda")
        row_s[:, at] = s.repeat_interleave(k, 1)
        out = dict(row_q=row_q[:rows].view(F8[case["q"]]), row_s=row_s[:, :rows].contiguous())
        if case["keep"]:
            out["q"], out["s"] = q, s
        return out
    y = torch.where(used[:, :, None], st["y"].float()[pos.clamp(min=0)], 0.0)
    out = (y * st["weight"][:, :, None]).sum(1).to(HP[case["x"]])
    if case["what"] == "combine":
        return out
    d = st["dout"].float()
    rows = st["y"].shape[0]
    dy = torch.zeros((rows + 1, case["cols"]), device="cuda")
    dy[torch.where(used, pos, rows).view(-1)] = (d[:, None, :] * st["weight"][:, :, None]).view(-1, case["cols"])
    return dict(out=out, dy=dy[:rows].to(HP[case["x"]]), dweight=(y * d[:, None, :]).sum(2))


def _plain_route(case, st):
    t, e, k = case["tokens"], case["experts"], case["k"]
    expert, has, p, w = _route(case, st["logits"], st["valid"])
    flat = torch.where(has, expert, e).view(-1)
    order = torch.sort(flat, stable=True).indices
    counts = torch.zeros(e + 1, dtype=torch.long, device="cuda").scatter_add_(0, flat, torch.ones_like(flat))[:e]
    offsets = torch.zeros(e + 1, dtype=torch.long, device="cuda")
    offsets[1:] = torch.cumsum(counts, 0)
    at = torch.arange(t * k, device="cuda")
    position = torch.empty_like(order)
    position[order] = at
    out = dict(expert=torch.where(has, expert, -1).int(), weight=w, offsets=offsets.int(), counts=counts.int(),
               position=torch.where(has, position.view(t, k), -1).int(),
               token=torch.where(at < offsets[-1], order // k, -1).int())
    if not case["grad"]:
        return out
    slope = counts * (e / (counts.sum().clamp(min=1) * has[:, 0].sum().clamp(min=1)))
    out["slope"], out["loss"] = slope.float(), (slope * p.sum(0)).sum().float().view(1)
    dw = torch.where(has, st["dweight"], 0.0)
    dp = (st["dloss"] * out["slope"]).expand(t, e)
    if case["normalize"]:
        total = torch.where(has, p.gather(1, expert), 0.0).sum(1, keepdim=True)
        dw = (dw - (dw * w).sum(1, keepdim=True)) / torch.where(has[:, :1], total, 1.0)
    dp = dp.scatter_add(1, expert, torch.where(has, dw, 0.0))
    out["dlogits"] = (p * (dp - (p * dp).sum(1, keepdim=True))).to(HP[case["x"]])
    return out


def _own(st):
    import fp8_delayed_scaling_gb300 as fd

    case = st["case"]
    op = case["op"]
    if op == "route":
        out = {n: st[n] for n in ("expert", "weight", "position", "token", "offsets", "counts")}
        if case["grad"]:
            out.update(slope=st["slope"], loss=st["loss"])
        fd.moe_route(st["logits"], **out, workspace=st["ws"], valid=st["valid"], normalize=case["normalize"])
        if case["grad"]:
            fd.moe_route_bwd(st["logits"], st["expert"], st["weight"], st["dlogits"], dweight=st["dweight"], slope=st["slope"],
                             dloss=st["dloss"], normalize=case["normalize"])
            out["dlogits"] = st["dlogits"]
        return out
    if op == "act":
        fmt = F8[case["q"]]
        fd.fp8_block_act(st["h"], ACT[case["act"]], CODE[case["q"]], st["g_q"], st["g_s"], h_q=st["h_q"], h_s=st["h_s"],
                         offsets=st["off"])
        out = dict(g_q=st["g_q"].view(fmt), g_s=st["g_s"])
        if case["keep"]:
            out.update(h_q=st["h_q"].view(fmt), h_s=st["h_s"])
        return out
    if op == "dact":
        fmt = F8[case["q"]]
        fd.fp8_block_dact(st["dg"], st["h_q"], fd.E4M3, st["h_s"], ACT[case["act"]], CODE[case["q"]], dh_q=st["dh_q"],
                          dh_s=st["dh_s"], dh_qt=st["dh_qt"], dh_st=st["dh_st"], g_qt=st["g_qt"], g_st=st["g_st"],
                          offsets=st["off"], dbias=st["db"], workspace=st["ws"])
        out = dict(dh_q=st["dh_q"].view(fmt), dh_s=st["dh_s"], dh_qt=st["dh_qt"].view(fmt), dh_st=st["dh_st"],
                   g_qt=st["g_qt"].view(F8["e4m3"]), g_st=st["g_st"])
        if case["dbias"]:
            out["dbias"] = st["db"]
        return out
    if op == "recode":
        fd.fp8_block_recode(st["q"], CODE[case["q"]], st["s"], CODE[case["to"]], st["col_q"], st["col_s"], offsets=st["off"],
                            index=st["index"])
        return dict(col_q=st["col_q"].view(F8[case["to"]]), col_s=st["col_s"])
    if case["what"] == "dispatch":
        fmt = F8[case["q"]]
        fd.fp8_block_dispatch(st["x"], CODE[case["q"]], st["position"], st["row_q"], st["row_s"], q=st["q"], s=st["s"])
        out = dict(row_q=st["row_q"].view(fmt), row_s=st["row_s"])
        if case["keep"]:
            out.update(q=st["q"].view(fmt), s=st["s"])
        return out
    fd.moe_combine(st["y"], st["position"], st["out"], weight=st["weight"])
    if case["what"] == "combine":
        return st["out"]
    fd.moe_combine_bwd(st["dout"], st["y"], st["position"], st["weight"], st["dy"], st["dweight"])
    return dict(out=st["out"], dy=st["dy"], dweight=st["dweight"])


# ------------------------------------------------------------------------------------------------ floors
def work(case):
    op = case["op"]
    if op == "route":
        t, e, k = case["tokens"], case["experts"], case["k"]
        esz = 2 if case["x"] == "bf16" else 4
        used = t - case["padded"]
        n = used * e * esz + t * k * 12 + used * k * 4 + 8 * e + (t if case["padded"] else 0)
        if case["grad"]:
            n += t * e * esz + used * k * 4 + 4 * e
        return dict(bytes=n, flops=used * e * (12 if case["grad"] else 4))
    esz = 2 if case.get("x") == "bf16" else 4
    if op in ("act", "dact"):
        r, c = max(0, case["rows"] - case["behind"]), case["cols"]
        wide = 2 * c if _gated(case) else c
        if op == "act":
            kept = wide if case["keep"] else 0
            return dict(bytes=r * (wide * esz + c + kept) + r * 4 * (_ceil(c, 128) + _ceil(kept, 128)) + 1, flops=12 * r * c)
        blocks = _ceil(r, 128)
        return dict(bytes=r * (c * esz + wide + 2 * wide + c) + 4 * r * 2 * _ceil(wide, 128) + 4 * blocks * (wide + c)
                    + (4 * wide if case["dbias"] else 0) + 1, flops=30 * r * c)
    if op == "recode":
        r, c = max(0, case["rows"] - case["behind"]), case["cols"]
        src = min(r, case["source"])
        return dict(bytes=(src + r) * c + 4 * src * _ceil(c, 128) + 4 * _ceil(r, 128) * c + (4 * r if case["index"] else 0) + 1, flops=4 * r * c)
    t, k, c = case["tokens"] - case["padded"], case["k"], case["cols"]
    n = 4 * case["tokens"] * k
    if case["what"] == "dispatch":
        copies = t * k + (case["tokens"] if case["keep"] else 0)
        read = case["tokens"] if case["keep"] else t
        return dict(bytes=n + read * c * esz + copies * (c + 4 * _ceil(c, 128)), flops=4 * t * c)
    n += 4 * t * k + t * k * c * esz + case["tokens"] * c * esz
    if case["what"] == "train":
        n += t * c * esz + t * k * c * esz + 4 * case["tokens"] * k
    return dict(bytes=n, flops=2 * t * k * c * (3 if case["what"] == "train" else 1))


# ------------------------------------------------------------------------------------------------ 64 bits
def _nearest(v, fmt):
    """The FP8 value nearest to v (fp64, within the format's range), ties to the even code, from the format's
    definition: mantissa bits p, smallest normal exponent lo."""
    p, lo = (3, -6) if fmt == "e4m3" else (2, -14)
    mag = v.abs()
    e = torch.floor(torch.log2(mag.clamp(min=2.0 ** -60))).clamp(min=lo)
    e = torch.where(mag < torch.exp2(e), (e - 1).clamp(min=lo), torch.where(mag >= torch.exp2(e + 1), e + 1, e))
    step = torch.exp2(e - p)
    return (torch.round(v / step) * step).clamp(-FP8_MAX[fmt], FP8_MAX[fmt])


def _blocks64(x, fmt):
    """Values x [blocks, 128 or so] in fp64: (code values, stored factors), each block on its own.  The scale, its
    reciprocal and the scaled value are defined as rounded to fp32."""
    top = x.abs().amax(1, keepdim=True)
    scale = torch.where(top > 0, (FP8_MAX[fmt] / top.clamp(min=TINY)).float().double(), 1.0)
    return _nearest((x * scale).float().double(), fmt), (1.0 / scale).float().double()[:, 0]


def _rows64(x, fmt, lo, hi):
    """Row-wise codes' values and factors of rows lo .. hi-1, zeros for the others."""
    q, s = torch.zeros_like(x), torch.zeros((_ceil(x.shape[1], 128), x.shape[0]), dtype=torch.float64, device="cuda")
    for b in range(s.shape[0] if hi > lo else 0):
        q[lo:hi, 128 * b:128 * b + 128], s[b, lo:hi] = _blocks64(x[lo:hi, 128 * b:128 * b + 128], fmt)
    return q, s


def _cols64(x, fmt, off):
    """Transposed codes' values and factors of the groups."""
    q = torch.zeros((x.shape[1], _capacity(x.shape[0], len(off) - 1)), dtype=torch.float64, device="cuda")
    s = torch.zeros((q.shape[1] // 128, x.shape[1]), dtype=torch.float64, device="cuda")
    at = 0
    for lo, hi in zip(off[:-1], off[1:]):
        for r in range(lo, hi, 128):
            part = x[r:min(r + 128, hi)].t()
            q[:, 128 * at:128 * at + part.shape[1]], s[at] = _blocks64(part, fmt)
            at += 1
    return q, s


def _decoded64(q, fmt, s):
    v = q.view(F8[fmt]).double()
    for b in range(s.shape[0]):
        v[:, 128 * b:128 * b + 128] *= s[b].double()[:, None]
    return v


def _act64(a, kind):
    """act(a) and its derivative from their definitions: GELU(a) = a Phi(a), SiLU(a) = a / (1 + e^-a)."""
    if kind in ("gelu", "geglu"):
        cdf = 0.5 * torch.special.erfc(-a / 2.0 ** 0.5)
        return a * cdf, cdf + a * torch.exp(-a * a / 2) / (2 * torch.pi) ** 0.5
    s = torch.sigmoid(a)
    return a * s, s + a * s * torch.sigmoid(-a)


def _route64(case, st):
    t, e, k = case["tokens"], case["experts"], case["k"]
    l = st["logits"].double().cpu()
    if st["valid"] is not None:
        l[~st["valid"].cpu()] = -torch.inf
    some = torch.isfinite(l).any(1)
    p = torch.zeros_like(l)
    p[some] = torch.softmax(l[some], 1)
    chosen = torch.zeros((t, e), dtype=torch.bool)
    pick, left = torch.full((t, k), -1), l.clone()
    for j in range(k):
        best = left.max(1).values
        first = (left == best[:, None]).int().argmax(1)  # the lowest of equal ones
        ok = best > -torch.inf
        pick[ok, j] = first[ok]
        chosen[ok, first[ok]] = True
        left[ok, first[ok]] = -torch.inf
    w = torch.where(pick >= 0, p.gather(1, pick.clamp(min=0)), 0.0)
    total = w.sum(1, keepdim=True)
    share = w / torch.where(total > 0, total, 1.0) if case["normalize"] else w
    out = dict(expert=None, weight=share, offsets=None, counts=None, position=None, token=None)
    if not case["grad"]:
        return out
    counts, n = chosen.sum(0).double(), int(some.sum())
    slope = e * counts / max(1.0, float(counts.sum())) / max(1, n)
    out["slope"], out["loss"] = slope, (slope * p.sum(0)).sum().view(1)
    dw = torch.where(pick >= 0, st["dweight"].double().cpu(), 0.0)
    if case["normalize"]:
        dw = torch.where(pick >= 0, (dw - (dw * share).sum(1, keepdim=True)) / torch.where(total > 0, total, 1.0), 0.0)
    dp = float(st["dloss"]) * slope.expand(t, e).clone()
    for j in range(k):
        ok = pick[:, j] >= 0
        dp[ok, pick[ok, j]] += dw[ok, j]
    out["dlogits"] = p * (dp - (p * dp).sum(1, keepdim=True))
    return out


def exact(case, seed):
    st, op = prepare(case, seed), case["op"]
    if op == "route":
        return _route64(case, st)
    if op in ("act", "dact", "recode"):
        off = st["off"].tolist() if st["off"] is not None else [0, case["rows"]]
    if op == "act":
        h, c = st["h"].double(), case["cols"]
        y = _act64(h[:, :c], case["act"])[0]
        out = dict(zip(("g_q", "g_s"), _rows64(y * h[:, c:] if _gated(case) else y, case["q"], off[0], off[-1])))
        if case["keep"]:
            out["h_q"], out["h_s"] = _rows64(h, case["q"], off[0], off[-1])
        return out
    if op == "dact":
        h, c, dg = _decoded64(st["h_q"], "e4m3", st["h_s"]), case["cols"], st["dg"].double()
        y, d = _act64(h[:, :c], case["act"])
        dh = dg * d
        if _gated(case):
            dh = torch.cat([dh * h[:, c:], dg * y], 1)
            y = y * h[:, c:]
        out = dict(zip(("dh_q", "dh_s"), _rows64(dh, case["q"], off[0], off[-1])))
        out["dh_qt"], out["dh_st"] = _cols64(dh, case["q"], off)
        out["g_qt"], out["g_st"] = _cols64(y, "e4m3", off)
        if case["dbias"]:
            out["dbias"] = dh.sum(0)
        return out
    if op == "recode":
        x = _decoded64(st["q"], case["q"], st["s"])
        return dict(zip(("col_q", "col_s"), _cols64(x if st["index"] is None else x[st["index"].long()], case["to"], off)))
    pos, k = st["position"].long(), case["k"]
    if case["what"] == "dispatch":
        q, s = _rows64(st["x"].double(), case["q"], 0, case["tokens"])
        row_q = torch.zeros((q.shape[0] * k, q.shape[1]), dtype=torch.float64, device="cuda")
        row_s = torch.zeros((s.shape[0], q.shape[0] * k), dtype=torch.float64, device="cuda")
        for j in range(k):
            t = (pos[:, j] >= 0).nonzero()[:, 0]
            row_q[pos[t, j]], row_s[:, pos[t, j]] = q[t], s[:, t]
        out = dict(row_q=row_q, row_s=row_s)
        if case["keep"]:
            out["q"], out["s"] = q, s
        return out
    y, w = st["y"].double(), st["weight"].double()
    out = torch.zeros((case["tokens"], case["cols"]), dtype=torch.float64, device="cuda")
    dy, dw = torch.zeros_like(y), torch.zeros_like(w)
    for j in range(k):
        t = (pos[:, j] >= 0).nonzero()[:, 0]
        out[t] += w[t, j, None] * y[pos[t, j]]
        if case["what"] == "train":
            dy[pos[t, j]] = w[t, j, None] * st["dout"][t].double()
            dw[t, j] = (y[pos[t, j]] * st["dout"][t].double()).sum(1)
    return out if case["what"] == "combine" else dict(out=out, dy=dy, dweight=dw)
