"""What the block-scaled FP8 operators are measured on.

Block scaling keeps one fp32 scale per 128 consecutive values along a product's reduction axis (activations
and gradients) or per 128 x 128 block (weights).  The operators: `quantize` (activations and gradients, row-wise
codes for the forward and dgrad products, transposed codes for the wgrad product, whole or per group of rows),
`weight` (128 x 128 blocks, codes and transposed codes), `gemm` (one product), `grouped` (the products of
ragged groups of tokens with their expert's weight) and `wgrad` (the ragged groups' weight gradients).

`own` is false: plain torch in fp32; true: the framework's entry points.
"""
import torch

own = False

F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FP8_MAX = {"e4m3": 448.0, "e5m2": 57344.0}
HP = {"bf16": torch.bfloat16, "fp32": torch.float32}
CODE = {"e4m3": 0, "e5m2": 1}
TINY = 2.0 ** -100  # a smaller block maximum counts as this one (its reciprocal stays finite)


def listed():
    return [
        # an activation of 8192 tokens at hidden 4096, quantised once for both the forward and the wgrad product
        dict(name="quantize 8192x4096", op="quantize", rows=8192, cols=4096, x="bf16", q="e4m3", groups=0, behind=0, dbias=False),
        # the gradient of an expert layer's output: E5M2, 2999 routed tokens over 24 experts, some rows unused
        dict(name="quantize 2999x1408 grouped", op="quantize", rows=2999, cols=1408, x="fp32", q="e5m2", groups=24, behind=100, dbias=False),
        # the fc1 weight of a 4096 -> 16384 MLP, after each optimizer step
        dict(name="weight 16384x4096", op="weight", mats=1, rows=16384, cols=4096, x="bf16"),
        # the weights of 32 small experts, from fp32 masters
        dict(name="weight 32x1008x2048", op="weight", mats=32, rows=1008, cols=2048, x="fp32"),
        # one new token through a square projection (latency)
        dict(name="gemm 1x4096x4096", op="gemm", m=1, n=4096, k=4096, a="e4m3", d="bf16", bias=False, b_rows=False),
        # a small decode batch through an up projection
        dict(name="gemm 37x11008x4096", op="gemm", m=37, n=11008, k=4096, a="e4m3", d="bf16", bias=True, b_rows=False),
        # the forward product of a large training step
        dict(name="gemm 16384x16384x4096", op="gemm", m=16384, n=16384, k=4096, a="e4m3", d="bf16", bias=True, b_rows=False),
        # a weight gradient over 8192 tokens (both operands scaled along the tokens), fp32 result
        dict(name="gemm 4096x11008x8192 rows", op="gemm", m=4096, n=11008, k=8192, a="e5m2", d="fp32", bias=False, b_rows=True),
        # decoding with experts: 128 routed rows over 64 experts, some of them idle
        dict(name="grouped 128 of 64", op="grouped", tokens=128, experts=64, n=2048, k=4096, a="e4m3", d="bf16", skew=1.0, behind=0),
        # training with experts: 32768 routed rows, uneven loads
        dict(name="grouped 32768 of 16", op="grouped", tokens=32768, experts=16, n=4096, k=2048, a="e4m3", d="bf16", skew=0.5, behind=64),
        # the weight gradients of the same layer
        dict(name="wgrad 32768 of 16", op="wgrad", tokens=32768, experts=16, n=4096, k=2048, a="e4m3", d="bf16", skew=0.5, behind=64),
        # the weight gradients of many small experts with few tokens each, fp32 result
        dict(name="wgrad 3001 of 48", op="wgrad", tokens=3001, experts=48, n=1408, k=2048, a="e5m2", d="fp32", skew=1.0, behind=0),
    ]


def _log(rng, lo, hi, step=1):
    """A size between lo and hi, spread over its logarithm, a multiple of step."""
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random() / step)) * step))


def draw(rng):
    op = rng.choice(["quantize", "weight", "gemm", "gemm", "grouped", "wgrad"])
    if op == "quantize":
        groups = rng.choice([0, rng.randint(1, 64)])
        return dict(op=op, rows=_log(rng, 1, 8192), cols=_log(rng, 256, 4096, 16), x=rng.choice(["bf16", "fp32"]),
                    q=rng.choice(["e4m3", "e5m2"]), groups=groups, behind=rng.randint(0, 70) if groups else 0,
                    dbias=not groups and rng.random() < 0.5)
    if op == "weight":
        return dict(op=op, mats=rng.choice([1, _log(rng, 2, 32)]), rows=_log(rng, 128, 2048, 16),
                    cols=_log(rng, 128, 4096, 16), x=rng.choice(["bf16", "fp32"]))
    if op == "gemm":
        rows = rng.random() < 0.3
        return dict(op=op, m=_log(rng, 256, 4096, 16) if rows else _log(rng, 1, 8192), n=_log(rng, 512, 12288, 16),
                    k=_log(rng, 512, 8192, 16), a=rng.choice(["e4m3", "e5m2"]), d=rng.choice(["bf16", "fp32"]),
                    bias=rng.random() < 0.5, b_rows=rows)
    return dict(op=op, tokens=_log(rng, 1 if op == "grouped" else 64, 16384), experts=_log(rng, 2, 64),
                n=_log(rng, 512, 2048, 16), k=_log(rng, 512, 4096, 16), a=rng.choice(["e4m3", "e5m2"]),
                d=rng.choice(["bf16", "fp32"]), skew=rng.choice([0.0, 0.5, 1.0]), behind=rng.randint(0, 70))


def _loads(tokens, experts, skew):
    """Tokens per expert, most loaded first: shares of 1 / (i + 1)^skew, rounded down, what is left to the first."""
    w = [1.0 / (i + 1) ** skew for i in range(experts)]
    n = [int(tokens * v / sum(w)) for v in w]
    n[0] += tokens - sum(n)
    return n


def _ceil(a, b):
    return (a + b - 1) // b


def _capacity(rows, groups):
    """Columns of the transposed codes: every group padded to a multiple of 128, at most this many in all."""
    return (rows + 127 * min(groups, rows)) // 128 * 128


# ------------------------------------------------------------------------------------------------ plain forms
def _scales(amax, fmt):
    """(scale, stored factor) of blocks with these maxima: scale = fp8_max / amax, factor = 1 / scale; 1 where a
    block holds nothing."""
    one = torch.ones_like(amax)
    scale = torch.where(amax > 0, (one * FP8_MAX[fmt]) / amax.clamp(min=TINY), one)  # tensor by tensor: a true division
    return scale, one / scale


def _magnitude(x):
    return torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x))


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
    scale, inv = _scales(_magnitude(xb).amax(2), fmt)
    return _codes(xb, scale[:, :, None], fmt).view(r, -1)[:, :c], inv.t().contiguous()


def _quantize_cols(x, fmt):
    """Along the rows, x's rows being a multiple of 128: transposed codes [C, R] and factors [R / 128, C]."""
    r, c = x.shape
    xb = x.float().view(-1, 128, c)
    scale, inv = _scales(_magnitude(xb).amax(1), fmt)
    return _codes(xb, scale[:, None, :], fmt).view(r, c).view(torch.uint8).t().contiguous().view(F8[fmt]), inv


def _quantize_blocks(w, fmt):
    """128 x 128 blocks of w [E, R, C]: codes and factors [E, C / 128, R / 128]."""
    e, r, c = w.shape
    wb = _pad128(_pad128(w.float(), 2), 1)
    wb = wb.view(e, wb.shape[1] // 128, 128, -1, 128)
    scale, inv = _scales(_magnitude(wb).amax((2, 4)), fmt)
    q = _codes(wb, scale[:, :, None, :, None], fmt).view(e, wb.shape[1] * 128, -1)
    return q[:, :r, :c].contiguous(), inv.transpose(1, 2).contiguous()


def _slots(off, rows, groups):
    """For each column of the padded, transposed codes: its row of x (rows where it has none)."""
    n = off[1:] - off[:-1]
    pad = torch.cumsum((n + 127) // 128 * 128, 0)
    at = torch.arange(_capacity(rows, groups), device=off.device)
    g = torch.searchsorted(pad, at, right=True)
    inside = g < groups
    g = g.clamp(max=groups - 1)
    k = at - (pad - (n + 127) // 128 * 128)[g]
    return torch.where(inside & (k < n[g]), off[:-1][g] + k, torch.full_like(at, rows)), inside


def _values(q, fmt, s, rows_per_scale):
    """The numbers that codes q [R, K] with factors s [K / 128, R / rows_per_scale] stand for."""
    r, k = q.shape
    f = s.t().repeat_interleave(rows_per_scale, 0)[:r].repeat_interleave(128, 1)[:, :k]
    return q.view(F8[fmt]).float() * f


def _product(a, b, bias, dtype):
    y = a @ b.t()
    return (y if bias is None else y + bias.float()).to(dtype)


# ------------------------------------------------------------------------------------------------ inputs
def _activation(rows, cols, g, dtype):
    """Normal values with a spread of channel sizes, as activations have."""
    ch = torch.exp(torch.randn(cols, device="cuda", generator=g) * 1.5)
    return (torch.randn((rows, cols), device="cuda", generator=g) * ch).to(dtype)


def _offsets(case, rows_total, groups, seed):
    n = _loads(rows_total - case["behind"], groups, case.get("skew", 0.7)) if rows_total > case["behind"] else [0] * groups
    order = torch.randperm(groups, generator=torch.Generator().manual_seed(seed))
    off = torch.zeros(groups + 1, dtype=torch.int32)
    off[1:] = torch.cumsum(torch.tensor(n, dtype=torch.int32)[order], 0)
    return off.cuda()


def _experts(n_mats, n, k, g):
    """Expert weights' codes and factors, made matrix by matrix where they are many."""
    q = torch.empty((n_mats, n, k), dtype=torch.uint8, device="cuda")
    s = torch.empty((n_mats, _ceil(k, 128), _ceil(n, 128)), device="cuda")
    for e in range(n_mats):
        w = torch.randn((1, n, k), device="cuda", generator=g) * 0.02
        a, b = _quantize_blocks(w, "e4m3")
        q[e], s[e] = a[0].view(torch.uint8), b[0]
    return q, s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    st, op = dict(case=case), case["op"]
    if op == "quantize":
        rows, cols, groups = case["rows"], case["cols"], case["groups"]
        st["x"] = _activation(rows, cols, g, HP[case["x"]])
        st["off"] = _offsets(case, rows, groups, seed) if groups else None
        cap = _capacity(rows, max(1, groups))
        u8 = dict(dtype=torch.uint8, device="cuda")
        st["row_q"], st["row_s"] = torch.zeros((rows, cols), **u8), torch.zeros((_ceil(cols, 128), rows), device="cuda")
        st["col_q"], st["col_s"] = torch.zeros((cols, cap), **u8), torch.zeros((cap // 128, cols), device="cuda")
        st["db"] = torch.zeros(cols, device="cuda") if case["dbias"] else None
        st["ws"] = torch.empty(_ceil(rows, 128) * cols * 4, **u8) if case["dbias"] else None
    elif op == "weight":
        e, r, c = case["mats"], case["rows"], case["cols"]
        st["w"] = (torch.randn((e, r, c), device="cuda", generator=g) * 0.02).to(HP[case["x"]])
        u8 = dict(dtype=torch.uint8, device="cuda")
        st["q"], st["s"] = torch.empty((e, r, c), **u8), torch.empty((e, _ceil(c, 128), _ceil(r, 128)), device="cuda")
        st["q_t"], st["s_t"] = torch.empty((e, c, r), **u8), torch.empty((e, _ceil(r, 128), _ceil(c, 128)), device="cuda")
    elif op == "gemm":
        m, n, k = case["m"], case["n"], case["k"]
        q, st["a_s"] = _quantize_rows(_activation(m, k, g, torch.bfloat16), case["a"])
        st["a"] = q.contiguous().view(torch.uint8)
        if case["b_rows"]:
            q, st["b_s"] = _quantize_rows(_activation(n, k, g, torch.bfloat16), "e4m3")
            st["b"] = q.contiguous().view(torch.uint8)
        else:
            q, s = _experts(1, n, k, g)
            st["b"], st["b_s"] = q[0], s[0]
        st["bias"] = torch.randn(n, device="cuda", generator=g).bfloat16() if case["bias"] else None
        st["d"] = torch.empty((m, n), dtype=HP[case["d"]], device="cuda")
    elif op == "grouped":
        rows, e, n, k = case["tokens"] + case["behind"], case["experts"], case["n"], case["k"]
        q, st["a_s"] = _quantize_rows(_activation(rows, k, g, torch.bfloat16), case["a"])
        st["a"] = q.contiguous().view(torch.uint8)
        st["b"], st["b_s"] = _experts(e, n, k, g)
        st["off"] = _offsets(case, rows, e, seed)
        st["d"] = torch.zeros((rows, n), dtype=HP[case["d"]], device="cuda")
    else:
        rows, e, n, k = case["tokens"] + case["behind"], case["experts"], case["n"], case["k"]
        st["off"] = _offsets(case, rows, e, seed)
        src, _ = _slots(st["off"].long(), rows, e)
        for name, cols, fmt in (("a", n, case["a"]), ("b", k, "e4m3")):
            x = _activation(rows + 1, cols, g, torch.bfloat16)
            x[rows] = 0
            q, st[name + "_s"] = _quantize_cols(x[src], fmt)
            st[name] = q.view(torch.uint8)
        st["d"] = torch.empty((e, n, k), dtype=HP[case["d"]], device="cuda")
    torch.cuda.synchronize()
    if "off" in st and st["off"] is not None:
        st["longest"] = int((st["off"][1:] - st["off"][:-1]).max())  # the plain forms' padded length
    return st


# ------------------------------------------------------------------------------------------------ one pass
def run(st):
    if own:
        return _own(st)
    case = st["case"]
    op = case["op"]
    if op == "quantize":
        x, fmt, off = st["x"].float(), case["q"], st["off"]
        rows = x.shape[0]
        q, s = _quantize_rows(x, fmt)
        if off is None:
            xp, inside = _pad128(x, 0), None
        else:
            src, inside = _slots(off.long(), rows, case["groups"])
            xp = torch.cat([x, torch.zeros_like(x[:1])])[src]
            used = torch.arange(rows, device=x.device) < off[-1]
            q = torch.where(used[:, None], q.view(torch.uint8), 0).view(F8[fmt])
            s = torch.where(used[None, :], s, 0.0)
        qt, s_t = _quantize_cols(xp, fmt)
        if inside is not None:
            s_t = torch.where(inside[::128][:, None], s_t, 0.0)
        out = dict(row_q=q, row_s=s, col_q=qt, col_s=s_t)
        if case["dbias"]:
            out["dbias"] = x.sum(0)
        return out
    if op == "weight":
        q, s = _quantize_blocks(st["w"], "e4m3")
        q_t = q.view(torch.uint8).transpose(1, 2).contiguous().view(F8["e4m3"])
        return dict(q=q, s=s, q_t=q_t, s_t=s.transpose(1, 2).contiguous())
    if op == "gemm":
        a = _values(st["a"], case["a"], st["a_s"], 1)
        b = _values(st["b"], "e4m3", st["b_s"], 1 if case["b_rows"] else 128)
        return _product(a, b, st["bias"], HP[case["d"]])
    off = st["off"].long()
    e, n, k, longest = case["experts"], case["n"], case["k"], max(1, st["longest"])
    at = off[:-1, None] + torch.arange(longest, device=off.device)[None, :]  # [E, longest] rows of each expert
    here = at < off[1:, None]
    if op == "grouped":
        rows = st["a"].shape[0]
        a = torch.cat([_values(st["a"], case["a"], st["a_s"], 1), torch.zeros((1, k), device="cuda")])
        s = st["b_s"].transpose(1, 2).repeat_interleave(128, 1)[:, :n].repeat_interleave(128, 2)[:, :, :k]
        b = st["b"].view(F8["e4m3"]).float() * s
        y = torch.bmm(a[torch.where(here, at, rows)], b.transpose(1, 2))
        d = torch.zeros((rows + 1, n), device="cuda")
        d[torch.where(here, at, rows)] = y
        return d[:rows].to(HP[case["d"]])
    length = off[1:] - off[:-1]
    start = torch.cumsum((length + 127) // 128 * 128, 0) - (length + 127) // 128 * 128
    cap = st["a"].shape[1]
    slot = torch.where(here, start[:, None] + torch.arange(longest, device=off.device)[None, :], cap)
    a = torch.nn.functional.pad(_values(st["a"], case["a"], st["a_s"], 1), (0, 1))
    b = torch.nn.functional.pad(_values(st["b"], "e4m3", st["b_s"], 1), (0, 1))
    return torch.bmm(a.t()[slot].transpose(1, 2), b.t()[slot]).to(HP[case["d"]])


def _own(st):
    import fp8_delayed_scaling_gb300 as fd

    case = st["case"]
    op = case["op"]
    if op == "quantize":
        fd.fp8_block_quantize(st["x"], CODE[case["q"]], row_q=st["row_q"], row_s=st["row_s"], col_q=st["col_q"],
                              col_s=st["col_s"], offsets=st["off"], dbias=st["db"], workspace=st["ws"])
        out = dict(row_q=st["row_q"].view(F8[case["q"]]), row_s=st["row_s"],
                   col_q=st["col_q"].view(F8[case["q"]]), col_s=st["col_s"])
        if case["dbias"]:
            out["dbias"] = st["db"]
        return out
    if op == "weight":
        fd.fp8_block_quantize_weight(st["w"], fd.E4M3, q=st["q"], s=st["s"], q_t=st["q_t"], s_t=st["s_t"])
        return dict(q=st["q"].view(F8["e4m3"]), s=st["s"], q_t=st["q_t"].view(F8["e4m3"]), s_t=st["s_t"])
    if op == "gemm":
        fd.fp8_block_gemm(st["a"], CODE[case["a"]], st["a_s"], st["b"], fd.E4M3, st["b_s"], st["d"], bias=st["bias"])
    elif op == "grouped":
        fd.fp8_block_gemm_grouped(st["a"], CODE[case["a"]], st["a_s"], st["b"], fd.E4M3, st["b_s"], st["off"], st["d"])
    else:
        fd.fp8_block_gemm_grouped_wgrad(st["a"], CODE[case["a"]], st["a_s"], st["b"], fd.E4M3, st["b_s"], st["off"],
                                        st["d"])
    return st["d"]


# ------------------------------------------------------------------------------------------------ floors
def work(case):
    op = case["op"]
    if op == "quantize":
        r, c = case["rows"], case["cols"]
        used = r - case["behind"] if r > case["behind"] else 0
        esz = 2 if case["x"] == "bf16" else 4
        return dict(bytes=used * c * (esz + 2) + 2 * 4 * _ceil(used * c, 128) + (4 * c if case["dbias"] else 0), flops=4 * used * c)
    if op == "weight":
        e, r, c = case["mats"], case["rows"], case["cols"]
        return dict(bytes=e * (r * c * ((2 if case["x"] == "bf16" else 4) + 2) + 2 * 4 * _ceil(r, 128) * _ceil(c, 128)), flops=4 * e * r * c)
    dsz = 2 if case["d"] == "bf16" else 4
    n, k = case["n"], case["k"]
    if op == "gemm":
        m = case["m"]
        sb = _ceil(k, 128) * (n if case["b_rows"] else _ceil(n, 128))
        return dict(bytes=m * k + n * k + 4 * (_ceil(k, 128) * m + sb) + m * n * dsz + (2 * n if case["bias"] else 0), flops=2 * m * n * k)
    loads = _loads(case["tokens"], case["experts"], case["skew"])
    t = sum(loads)
    if op == "grouped":
        busy = sum(v > 0 for v in loads)
        return dict(bytes=t * k + busy * n * k + 4 * _ceil(k, 128) * (t + busy * _ceil(n, 128)) + t * n * dsz, flops=2 * t * n * k)
    blocks = sum(_ceil(v, 128) for v in loads)
    return dict(bytes=t * (n + k) + 4 * blocks * (n + k) + case["experts"] * n * k * dsz, flops=2 * t * n * k)


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


def _decoded64(q, fmt, s, per):
    """Codes q [R, K] (bytes) and factors s [K / 128, R / per] to fp64, block by block."""
    v = q.view(F8[fmt]).double()
    for b in range(s.shape[0]):
        f = s[b].double()
        v[:, 128 * b:128 * b + 128] *= (f if per == 1 else f.repeat_interleave(per)[:q.shape[0]])[:, None]
    return v


def exact(case, seed):
    op = case["op"]
    if op == "gemm" and 2.0 * case["m"] * case["n"] * case["k"] > 4e12:
        return None
    st = prepare(case, seed)
    if op == "quantize":
        x, fmt = st["x"].double(), case["q"]
        rows, cols = x.shape
        off = st["off"].tolist() if st["off"] is not None else [0, rows]
        q, s = torch.zeros_like(x), torch.zeros((_ceil(cols, 128), rows), dtype=torch.float64, device="cuda")
        for b in range(s.shape[0]):
            q[:off[-1], 128 * b:128 * b + 128], s[b, :off[-1]] = _blocks64(x[:off[-1], 128 * b:128 * b + 128], fmt)
        qt = torch.zeros((cols, _capacity(rows, max(1, case["groups"]))), dtype=torch.float64, device="cuda")
        st_ = torch.zeros((qt.shape[1] // 128, cols), dtype=torch.float64, device="cuda")
        block = 0
        for lo, hi in zip(off[:-1], off[1:]):
            for r in range(lo, hi, 128):
                part = x[r:min(r + 128, hi)].t()
                qt[:, 128 * block:128 * block + part.shape[1]], st_[block] = _blocks64(part, fmt)
                block += 1
        out = dict(row_q=q, row_s=s, col_q=qt, col_s=st_)
        if case["dbias"]:
            out["dbias"] = x.sum(0)
        return out
    if op == "weight":
        w = st["w"].double()
        e, r, c = w.shape
        q, s = torch.empty_like(w), torch.empty((e, _ceil(c, 128), _ceil(r, 128)), dtype=torch.float64, device="cuda")
        for i in range(s.shape[2]):
            for j in range(s.shape[1]):
                part = w[:, 128 * i:128 * i + 128, 128 * j:128 * j + 128]
                a, b = _blocks64(part.reshape(e, -1), "e4m3")
                q[:, 128 * i:128 * i + 128, 128 * j:128 * j + 128], s[:, j, i] = a.view(part.shape), b
        return dict(q=q, s=s, q_t=q.transpose(1, 2).contiguous(), s_t=s.transpose(1, 2).contiguous())
    if op == "gemm":
        y = _decoded64(st["a"], case["a"], st["a_s"], 1) @ _decoded64(st["b"], "e4m3", st["b_s"], 1 if case["b_rows"] else 128).t()
        return y + st["bias"].double() if case["bias"] else y
    off = st["off"].tolist()
    if op == "grouped":
        a = _decoded64(st["a"], case["a"], st["a_s"], 1)
        d = torch.zeros((a.shape[0], case["n"]), dtype=torch.float64, device="cuda")
        for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
            if hi > lo:
                d[lo:hi] = a[lo:hi] @ _decoded64(st["b"][e], "e4m3", st["b_s"][e], 128).t()
        return d
    a, b = _decoded64(st["a"], case["a"], st["a_s"], 1), _decoded64(st["b"], "e4m3", st["b_s"], 1)
    d = torch.zeros((case["experts"], case["n"], case["k"]), dtype=torch.float64, device="cuda")
    at = 0
    for e, (lo, hi) in enumerate(zip(off[:-1], off[1:])):
        d[e] = a[:, at:at + hi - lo] @ b[:, at:at + hi - lo].t()
        at += _ceil(hi - lo, 128) * 128
    return d
