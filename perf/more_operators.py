"""What is measured of the FP8 expert layer's operators: the root-mean-square norm
before the layer and its gradient, the block quantisation between the experts'
products, the gradient of SwiGLU from an 8-bit checkpoint, and the experts' products
of E4M3 codes with a scale for every 128 columns.

Each operator is computed in two ways on the same inputs: in its plain form, with
elementary torch operations in float32 (own = False), and by the calls of
combine_ep_route_topk_gb300 (own = True).  exact() computes it once more from its
definition in 64 bits.

  norm         ep_rms_norm             residual's addition, norm, rows and codes
  norm_grad    ep_rms_norm_backward    gradients of the rows and of the weight
  quant        ep_quantize_blocks      rows (or SwiGLU of rows) to E4M3, and the
               ep_dequantize_blocks    values that the codes stand for
  swiglu_grad  ep_swiglu_backward      from the rows or from their 8-bit checkpoint
  matmul       ep_expert_matmul_fp8    E4M3 rows x E4M3 expert weights, block scales
"""
import math

import torch

own = False

EPS = 1e-6
BLOCK = 128


def listed():
    return [
        # One sequence decodes one token: the norm before the gate is all latency.
        dict(name="norm 1 token", op="norm", rows=1, cols=7168, residual=True, y=True, codes=True,
             dtype="bf16", weight="bf16"),
        # Prefill of 8 x 4096 tokens: rows for the router, codes for the experts.
        dict(name="norm prefill", op="norm", rows=32768, cols=7168, residual=True, y=True,
             codes=True, dtype="bf16", weight="bf16"),
        # The training step of the prefill-sized norm: a gradient also comes along the residual.
        dict(name="norm gradient prefill", op="norm_grad", rows=32768, cols=7168, residual=True,
             dtype="bf16", weight="f32"),
        # A ragged batch of an odd number of float32 rows.
        dict(name="norm gradient odd", op="norm_grad", rows=5003, cols=2880, residual=False,
             dtype="f32", weight="f32"),
        # One token's 8 picks, between the experts' two products.
        dict(name="quantize swiglu 1 token", op="quant", rows=8, cols=2048, act="swiglu",
             keep=False, dtype="bf16"),
        # Prefill: the same for one GPU's rows, which also keeps the first product's output as
        # codes for the backward pass.
        dict(name="quantize swiglu checkpoint", op="quant", rows=32768, cols=2048, act="swiglu",
             keep=True, dtype="bf16"),
        # The backward pass of those rows from the checkpoint.
        dict(name="swiglu gradient checkpoint", op="swiglu_grad", rows=32768, cols=2048,
             saved="codes", dtype="bf16"),
        # The gradient from rows that were kept whole, an odd number of them.
        dict(name="swiglu gradient odd", op="swiglu_grad", rows=5003, cols=1440, saved="rows",
             dtype="bf16"),
        # One token's 8 picks on a GPU with 32 experts: the first product reads 8 experts' weights.
        dict(name="experts 1 token", op="matmul", rows=8, E=32, Nc=4096, Kd=7168, layout="contig",
             cap=0, gather=True, tokens=1, skew=0.0, out="bf16"),
        # Decode of 8 x 128 sequences, the share of one GPU of eight: masked rows, capacity 128.
        dict(name="experts decode masked", op="matmul", rows=1024, E=32, Nc=4096, Kd=7168,
             layout="masked", cap=128, gather=True, tokens=1024, skew=0.0, out="bf16"),
        # Prefill of 8 x 4096 tokens, one GPU's share of the first product, rows as dispatched.
        dict(name="experts prefill", op="matmul", rows=32768, E=32, Nc=4096, Kd=7168,
             layout="contig", cap=0, gather=False, tokens=0, skew=0.0, out="bf16"),
        # The second product of a 128-expert layer whose experts' popularity falls off steeply:
        # some experts get thousands of rows, some none; the last block of K is short.
        dict(name="experts skewed", op="matmul", rows=16384, E=128, Nc=2880, Kd=1440,
             layout="contig", cap=0, gather=False, tokens=0, skew=1.2, out="f32"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = _draw(rng)
        if c["op"] == "matmul":
            blocks = 0 if c["layout"] == "masked" else _blocks(c["rows"], c["E"])[1]
            if work(c)["flops"] > 1.9e12 or c["E"] * c["Nc"] * c["Kd"] > 9.4e8 \
                    or blocks * c["Nc"] * c["Kd"] > 8.5e9:
                continue
        return c


def _draw(rng):
    op = rng.choice(["norm", "norm_grad", "quant", "swiglu_grad", "matmul", "matmul"])
    if op != "matmul":
        cols = 16 * _log_int(rng, 4, 448)
        wide = cols if op in ("norm", "norm_grad") else 2 * cols
        c = dict(op=op, rows=_log_int(rng, 1, min(65536, 134217728 // wide)), cols=cols,
                 dtype=rng.choice(["bf16", "bf16", "f32"]))
        if op in ("norm", "norm_grad"):
            c.update(residual=rng.random() < 0.7, weight=rng.choice(["bf16", "f32"]))
        if op == "norm":
            outs = rng.choice([(True, True), (True, False), (False, True)])
            c.update(y=outs[0], codes=outs[1])
        if op == "quant":
            c["act"] = rng.choice(["none", "swiglu"])
            c["keep"] = c["act"] == "swiglu" and rng.random() < 0.5
        if op == "swiglu_grad":
            c["saved"] = rng.choice(["codes", "codes", "rows"])
        return c
    E = _log_int(rng, 1, 128)
    c = dict(op=op, rows=_log_int(rng, 1, 32768), E=E, Nc=_log_int(rng, 64, 7168),
             Kd=16 * _log_int(rng, 8, 448), layout=rng.choice(["contig", "contig", "masked"]),
             cap=0, gather=rng.random() < 0.5, tokens=0, skew=rng.choice([0.0, 0.0, 0.8, 1.2]),
             out=rng.choice(["bf16", "bf16", "f32"]))
    if c["layout"] == "masked":
        c["cap"] = max(1, min(32768 // E, int(c["rows"] * rng.choice([1.1, 1.5, 3.0]) / E) + 1))
    if c["gather"]:
        c["tokens"] = max(1, c["rows"] // rng.choice([1, 2, 4]))
    return c


# ---- inputs -----------------------------------------------------------------------------------


def _dtype(name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _kb(cols):
    return -(-cols // BLOCK)


def _activations(rows, cols, g, dt):
    """Rows of different loudness with a few loud columns; made in pieces."""
    out = torch.empty((rows, cols), dtype=dt, device="cuda")
    loud = 1.0 + 6.0 * (torch.rand((1, cols), generator=g, device="cuda") < 0.01).float()
    step = max(1, (1 << 27) // cols)
    for i in range(0, rows, step):
        n = min(step, rows - i)
        x = torch.randn((n, cols), generator=g, device="cuda")
        x *= 0.5 + torch.rand((n, 1), generator=g, device="cuda")
        out[i:i + n] = x.mul_(loud)
    return out


def _codes(shape, sigma, g):
    """E4M3 codes of normally distributed values, as bytes."""
    out = torch.empty(shape, dtype=torch.uint8, device="cuda")
    flat = out.view(-1)
    step = 1 << 27
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        r = torch.randn((n,), generator=g, device="cuda").mul_(sigma).clamp_(-448.0, 448.0)
        flat[i:i + n] = r.to(torch.float8_e4m3fn).view(torch.uint8)
    return out


def _prepare_matmul(case, g):
    rows, E, Nc, Kd, cap = (case[k] for k in ("rows", "E", "Nc", "Kd", "cap"))
    pop = torch.arange(1, E + 1, device="cuda", dtype=torch.float32) ** -case["skew"]
    pop = pop[torch.randperm(E, generator=g, device="cuda")]
    picks = torch.multinomial(pop, rows, replacement=True, generator=g)
    counts = torch.bincount(picks, minlength=E)
    offs = torch.zeros((E + 1,), dtype=torch.int32, device="cuda")
    offs[1:] = torch.cumsum(counts, 0)
    out_rows = E * cap if case["layout"] == "masked" else rows
    xr = case["tokens"] if case["gather"] else out_rows
    # a block's largest of 128 (of 16384) normal values lies near 2.8 (4.2) sigma, which the
    # scale sends to 448
    st = dict(case, offs=offs, x=_codes((xr, Kd), 160.0, g), w=_codes((E, Nc, Kd), 106.0, g))
    st["xs"] = (0.5 + torch.rand((xr, _kb(Kd)), generator=g, device="cuda")) / 160.0
    st["ws"] = (0.5 + torch.rand((E, _kb(Nc), _kb(Kd)), generator=g, device="cuda")) \
        / (106.0 * math.sqrt(Kd))
    st["row_src"] = None
    if case["gather"]:
        st["row_src"] = torch.randint(0, xr, (rows,), generator=g, device="cuda",
                                      dtype=torch.int32)
    # rows of the masked buffer that belong to no token are not written: they stay zero
    st["y"] = torch.zeros((out_rows, Nc), dtype=_dtype(case["out"]), device="cuda")
    return st


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op = case["op"]
    if op == "matmul":
        return _prepare_matmul(case, g)
    rows, cols, dt = case["rows"], case["cols"], _dtype(case["dtype"])
    st = dict(case)
    if op in ("norm", "norm_grad"):
        st["weight"] = (1.0 + 0.2 * torch.randn((cols,), generator=g, device="cuda")) \
            .to(_dtype(case["weight"]))
        st["x"] = _activations(rows, cols, g, dt)
    if op == "norm":
        st["res"] = _activations(rows, cols, g, dt) if case["residual"] else None
    elif op == "norm_grad":
        st["d_y"] = _activations(rows, cols, g, dt).mul_(1e-2)
        st["d_res"] = _activations(rows, cols, g, dt).mul_(1e-2) if case["residual"] else None
        # what the forward pass kept, the rows that were normalised and their statistic
        v = st["x"].double().square_().mean(-1).add_(EPS)
        st["rstd"] = v.rsqrt().float()
    elif op == "quant":
        st["x"] = _activations(rows, 2 * cols if case["act"] == "swiglu" else cols, g, dt)
    else:
        st["d_act"] = _activations(rows, cols, g, dt).mul_(1e-2)
        st["x"] = _activations(rows, 2 * cols, g, dt)
        st["xs"] = None
        if case["saved"] == "codes":
            q, st["xs"] = _quantize(st["x"].float())
            st["x"] = q.view(torch.uint8)
    return st


# ---- plain forms ------------------------------------------------------------------------------


def _blocked(v):
    """Rows as blocks of 128 columns, the last one filled up with zeros."""
    pad = -v.shape[-1] % BLOCK
    if pad:
        v = torch.nn.functional.pad(v, (0, pad))
    return v.reshape(*v.shape[:-1], -1, BLOCK)


def _quantize(v):
    """float32 rows -> (E4M3 codes, scales)."""
    b = _blocked(v)
    top = b.abs().amax(-1)
    scale = torch.where(top > 0, top / 448.0, 1.0)
    codes = (b / scale[..., None]).to(torch.float8_e4m3fn)
    return codes.reshape(v.shape[0], -1)[:, :v.shape[1]].contiguous(), scale


def _restore(codes, scale):
    v = _blocked(codes.float()) * scale[..., None]
    return v.reshape(codes.shape[0], -1)[:, :codes.shape[1]]


def _norm_plain(st):
    z = st["x"]
    out = {}
    if st["res"] is not None:
        z = out["residual"] = (z.float() + st["res"].float()).to(z.dtype)
    f = z.float()
    rstd = 1.0 / torch.sqrt((f * f).mean(-1) + EPS)
    y = f * rstd[:, None] * st["weight"].float()
    out["rstd"] = rstd
    if st["y"]:
        out["y"] = y.to(z.dtype)
    if st["codes"]:
        codes, out["scales"] = _quantize(y)
        out["values"] = _restore(codes, out["scales"]).to(torch.bfloat16)
    return out


def _norm_grad_plain(st):
    dy, xh = st["d_y"].float(), st["x"].float() * st["rstd"][:, None]
    g = dy * st["weight"].float()
    dx = (g - xh * (g * xh).mean(-1, keepdim=True)) * st["rstd"][:, None]
    if st["d_res"] is not None:
        dx = dx + st["d_res"].float()
    return dx.to(st["x"].dtype), (dy * xh).sum(0)


def _quant_plain(st):
    x = st["x"].float()
    v = x
    if st["act"] == "swiglu":
        a, b = x[:, :st["cols"]], x[:, st["cols"]:]
        v = a / (1.0 + torch.exp(-a)) * b
    codes, scales = _quantize(v)
    out = [_restore(codes, scales).to(torch.bfloat16), scales]
    if st["keep"]:
        codes, scales = _quantize(x)
        out += [_restore(codes, scales).to(torch.bfloat16), scales]
    return out


def _swiglu_grad_plain(st):
    x = st["x"].float() if st["xs"] is None else \
        _restore(st["x"].view(torch.float8_e4m3fn), st["xs"])
    a, b, d = x[:, :st["cols"]], x[:, st["cols"]:], st["d_act"].float()
    s = 1.0 / (1.0 + torch.exp(-a))
    da = d * b * s * (1.0 + a * (1.0 - s))
    return torch.cat([da, d * (a * s)], -1).to(st["d_act"].dtype)


def _blocks(rows, E):
    """Rows of one block of the plain product, and how many blocks there can be."""
    if rows <= 64:
        return 1, rows
    return 128, rows // 128 + min(E, rows)


def _matmul_plain(st):
    E, cap, offs, y = st["E"], st["cap"], st["offs"].long(), st["y"]
    counts = offs[1:] - offs[:-1]
    w, ws = st["w"], st["ws"]
    if st["layout"] == "masked":
        slot = torch.arange(cap, device=y.device)
        valid = slot[None, :] < counts[:, None]
        out_row = torch.arange(E, device=y.device)[:, None] * cap + slot[None, :]
        src = offs[:-1, None] + slot[None, :] if st["gather"] else out_row
    else:
        B, nb = _blocks(st["rows"], E)
        ends = torch.cumsum((counts + B - 1) // B, 0)
        b = torch.arange(nb, device=y.device)
        e = torch.searchsorted(ends, b, right=True).clamp(max=E - 1)
        begin = offs[e] + (b - ends[e] + (counts[e] + B - 1) // B) * B
        out_row = begin[:, None] + torch.arange(B, device=y.device)[None, :]
        valid = (out_row < offs[e + 1][:, None]) & (b < ends[-1])[:, None]
        src = out_row
        w, ws = w[e], ws[e]
    if st["gather"]:
        src = st["row_src"].long()[src.clamp(max=st["rows"] - 1)]
    src = torch.where(valid, src, 0)
    w = _blocked(w.view(torch.float8_e4m3fn).float())
    w.mul_(ws[:, torch.arange(st["Nc"], device=y.device) // BLOCK][..., None])
    x = _blocked(st["x"].view(torch.float8_e4m3fn).float()[src]) * st["xs"][src][..., None]
    acc = torch.bmm(x.flatten(2), w.flatten(2).transpose(1, 2))
    # a block's rows past its expert's end go to one more row, which is dropped
    ext = torch.cat([y, y[:1]])
    ext[torch.where(valid, out_row, y.shape[0]).view(-1)] = acc.view(-1, acc.shape[-1]).to(y.dtype)
    return ext[:-1]


# ---- the framework's calls --------------------------------------------------------------------


def _run_own(st):
    import combine_ep_route_topk_gb300 as ep
    op = st["op"]
    if op == "norm":
        out = ep.alloc_norm(st["rows"], st["cols"], st["x"].dtype, st["x"].device, y=st["y"],
                            residual=st["res"] is not None, codes=st["codes"], rstd=True)
        ep.ep_rms_norm(st["x"], st["weight"], residual=st["res"], eps=EPS, out=out)
        got = {"rstd": out.rstd}
        if st["res"] is not None:
            got["residual"] = out.residual
        if st["y"]:
            got["y"] = out.y
        if st["codes"]:  # compared as the values that the codes stand for
            got["scales"] = out.scales
            got["values"] = ep.ep_dequantize_blocks(out.q, out.scales)
        return got
    if op == "norm_grad":
        return ep.ep_rms_norm_backward(st["d_y"], st["x"], st["weight"], st["rstd"],
                                       d_residual=st["d_res"])
    if op == "quant":
        swiglu = st["act"] == "swiglu"
        rows, wide = st["x"].shape
        x_q = x_scales = None
        if st["keep"]:
            x_q = torch.empty((rows, wide), dtype=torch.uint8, device="cuda")
            x_scales = torch.empty((rows, _kb(wide)), dtype=torch.float32, device="cuda")
        q, scales = ep.ep_quantize_blocks(st["x"], act=ep.EP_ACT_SWIGLU if swiglu else
                                          ep.EP_ACT_NONE, x_q=x_q, x_scales=x_scales)
        out = [ep.ep_dequantize_blocks(q, scales), scales]
        if st["keep"]:
            out += [ep.ep_dequantize_blocks(x_q, x_scales), x_scales]
        return out
    if op == "swiglu_grad":
        return ep.ep_swiglu_backward(st["d_act"], st["x"], x_scales=st["xs"])
    return ep.ep_expert_matmul_fp8(
        st["x"], st["xs"], st["w"], st["ws"], st["offs"],
        layout=ep.EP_LAYOUT_MASKED if st["layout"] == "masked" else ep.EP_LAYOUT_CONTIG,
        cap=st["cap"], row_src=st["row_src"], out=st["y"])


def run(state):
    if own:
        return _run_own(state)
    return {"norm": _norm_plain, "norm_grad": _norm_grad_plain, "quant": _quant_plain,
            "swiglu_grad": _swiglu_grad_plain, "matmul": _matmul_plain}[state["op"]](state)


# ---- what a pass cannot do without ------------------------------------------------------------


def work(case):
    op = case["op"]
    if op == "matmul":
        rows, E, Nc, Kd = case["rows"], case["E"], case["Nc"], case["Kd"]
        size = 4 if case["out"] == "f32" else 2
        share = [i ** -case["skew"] for i in range(1, E + 1)]
        total = sum(share)
        used = sum(1.0 - (1.0 - s / total) ** rows for s in share)  # experts that get any row
        if case["layout"] == "masked":
            rows = sum(min(case["cap"], rows * s / total) for s in share)
        xr = min(case["tokens"], rows) if case["gather"] else rows
        return {"bytes": used * (Nc * Kd + 4 * _kb(Nc) * _kb(Kd)) + xr * (Kd + 4 * _kb(Kd))
                + rows * (Nc * size + 4 * case["gather"]),
                "flops": 2.0 * rows * Nc * Kd}
    n, size = case["rows"] * case["cols"], 4 if case["dtype"] == "f32" else 2
    rows = 4 * case["rows"]
    # codes and scales written, read again and written as values
    coded = n * 4 + 2 * rows * _kb(case["cols"])
    if op == "norm":
        return {"bytes": n * size * (1 + 2 * case["residual"] + case["y"]) + rows
                + coded * case["codes"] + case["cols"] * (4 if case["weight"] == "f32" else 2),
                "flops": 6 * n}
    if op == "norm_grad":
        return {"bytes": n * size * (3 + case["residual"]) + rows
                + case["cols"] * (8 if case["weight"] == "f32" else 6), "flops": 11 * n}
    if op == "quant":
        wide = 2 if case["act"] == "swiglu" else 1
        return {"bytes": n * wide * size + coded
                + (2 * n * 4 + 2 * rows * _kb(2 * case["cols"])) * case["keep"],
                "flops": 6 * n * wide}
    kept = 2 * n + rows * _kb(2 * case["cols"]) if case["saved"] == "codes" else 2 * n * size
    return {"bytes": 3 * n * size + kept, "flops": 14 * n}


# ---- 64 bits ----------------------------------------------------------------------------------


def _e4m3_64(v):
    """The nearest E4M3 value, ties to the even code, of values within 448 of zero."""
    _, ex = torch.frexp(v)  # |v| = m 2^ex with m in [1/2, 1): 3 bits behind the leading one
    step = torch.ldexp(torch.ones_like(v), (ex - 4).clamp(min=-9))
    return (v / step).round() * step


def _coded64(v):
    """The values that a block quantisation of v keeps, and its scales."""
    rows, cols = v.shape
    out, scales = torch.empty_like(v), []
    for c in range(0, cols, BLOCK):
        b = v[:, c:c + BLOCK]
        top = b.abs().max(-1, keepdim=True).values
        s = (top / 448).masked_fill(top == 0, 1.0)
        out[:, c:c + BLOCK] = _e4m3_64(b / s) * s
        scales.append(s)
    return out, torch.cat(scales, -1)


def _values64(codes, scales):
    rep = scales.double().repeat_interleave(BLOCK, -1)[..., :codes.shape[-1]]
    return codes.view(torch.float8_e4m3fn).to(torch.float64) * rep


def _exact_norm(case, st):
    x = st["x"].double()
    out = {}
    if case["residual"]:
        # the sum as the residual stream carries it, in the rows' own type
        x = (x + st["res"].double()).to(st["x"].dtype).double()
        out["residual"] = x
    r = (x.square().sum(-1) / case["cols"] + EPS).sqrt().reciprocal()
    y = x * r.unsqueeze(-1) * st["weight"].double()
    out["rstd"] = r
    if case["y"]:
        out["y"] = y
    if case["codes"]:
        out["values"], out["scales"] = _coded64(y)
    return out


def _exact_norm_grad(case, st):
    x, r = st["x"].double(), st["rstd"].double().unsqueeze(-1)
    up = st["d_y"].double()
    dw = (up * x * r).sum(0)
    up = up * st["weight"].double()
    # y = x r(x) w with dr/dx = -r^3 x / cols
    dx = up * r - x * r ** 3 * ((up * x).sum(-1, keepdim=True) / case["cols"])
    if case["residual"]:
        dx = dx + st["d_res"].double()
    return dx, dw


def _exact_quant(case, st):
    x = st["x"].double()
    v = x
    if case["act"] == "swiglu":
        g = x[:, :case["cols"]]
        v = g * torch.sigmoid(g) * x[:, case["cols"]:]
    out = list(_coded64(v))
    return out + list(_coded64(x)) if case["keep"] else out


def _exact_swiglu_grad(case, st):
    x = st["x"].double() if case["saved"] == "rows" else _values64(st["x"], st["xs"])
    g, u, d = x[:, :case["cols"]], x[:, case["cols"]:], st["d_act"].double()
    p, q = torch.sigmoid(g), torch.sigmoid(-g)
    return torch.cat([d * u * (p + g * p * q), d * g * p], -1)


def _exact_matmul(case, st):
    out = st["y"].double()
    offs = st["offs"].tolist()
    for e in range(case["E"]):
        lo, hi = offs[e], offs[e + 1]
        if case["layout"] == "masked":
            hi = min(hi, lo + case["cap"])
        if lo == hi:
            continue
        to = e * case["cap"] if case["layout"] == "masked" else lo
        at = st["row_src"][lo:hi].long() if case["gather"] else \
            torch.arange(to, to + hi - lo, device="cuda")
        per_row = st["ws"][e].repeat_interleave(BLOCK, 0)[:case["Nc"]]
        out[to:to + hi - lo] = _values64(st["x"][at], st["xs"][at]) \
            @ _values64(st["w"][e], per_row).T
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "quant": _exact_quant,
            "swiglu_grad": _exact_swiglu_grad, "matmul": _exact_matmul}[case["op"]](case, st)
