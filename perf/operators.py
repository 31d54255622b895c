"""What is measured of the expert operators: the gate and its gradient, the
8-bit quantisation of activation rows, and the experts' 8-bit products.

Each operator is computed in two ways on the same inputs: in its plain form,
with elementary torch operations in float32 (own = False), and by the calls of
combine_ep_route_topk_gb300 (own = True).  exact() computes it once more from
its definition in 64 bits.

  gate       ep_gate_topk           scores, balance bias, groups, top-K, weights
  gate_grad  ep_gate_topk_backward  gradient of the weights to the logits
  quant      ep_quantize_rows       rows (or SwiGLU of rows) to int8 + row scale
  matmul     ep_expert_matmul       int8 rows x int8 expert weights, two scales
"""
import math

import torch

own = False

SIGMOID, SOFTMAX = "sigmoid", "softmax"
F32_MAX = 3.4028234663852886e38


def listed():
    return [
        # One sequence decodes one token: the gate of a 256-expert layer is all latency.
        dict(name="gate 1 token", op="gate", N=1, E=256, K=8, score=SIGMOID, bias=True, groups=8,
             topk_groups=4, group_top=2, renorm=True, scale=2.5, dtype="f32", masked=0.0),
        # The decode step of 8 x 128 sequences, logits as the bf16 product before it left them.
        dict(name="gate decode", op="gate", N=1024, E=256, K=8, score=SIGMOID, bias=True,
             groups=8, topk_groups=4, group_top=2, renorm=True, scale=2.5, dtype="bf16",
             masked=0.0),
        # Prefill of 8 x 4096 tokens: the largest gate call.
        dict(name="gate prefill", op="gate", N=32768, E=256, K=8, score=SIGMOID, bias=True,
             groups=8, topk_groups=4, group_top=2, renorm=True, scale=2.5, dtype="f32",
             masked=0.0),
        # A softmax gate of an odd number of experts over a ragged batch; a tenth of the experts
        # is masked out per token, and some tokens have none left.
        dict(name="gate odd softmax", op="gate", N=5003, E=61, K=6, score=SOFTMAX, bias=False,
             groups=1, topk_groups=1, group_top=1, renorm=False, scale=1.0, dtype="f32",
             masked=0.1),
        # The training step of the prefill-sized gate.
        dict(name="gate gradient sigmoid", op="gate_grad", N=32768, E=256, K=8, score=SIGMOID,
             renorm=True, scale=2.5, dtype="f32", masked=0.0),
        # Without renormalised weights the softmax sends a gradient to every expert's logit.
        dict(name="gate gradient softmax", op="gate_grad", N=4999, E=128, K=4, score=SOFTMAX,
             renorm=False, scale=1.0, dtype="bf16", masked=0.05),
        # The tokens of a decode step, quantised before the experts' first product.
        dict(name="quantize decode", op="quant", rows=1024, cols=7168, act="none", dtype="bf16"),
        # Between the experts' two products of a prefill: SwiGLU and quantisation in one pass.
        dict(name="quantize swiglu prefill", op="quant", rows=32768, cols=2048, act="swiglu",
             dtype="bf16"),
        # One token's 8 picks on a GPU with 32 experts: the first product reads 8 experts' weights.
        dict(name="experts 1 token", op="matmul", rows=8, E=32, Nc=4096, Kd=7168, layout="contig",
             cap=0, gather=True, tokens=1, skew=0.0, out="bf16"),
        # Decode of 8 x 128 sequences, the share of one GPU of eight: masked rows, capacity 128.
        dict(name="experts decode masked", op="matmul", rows=1024, E=32, Nc=4096, Kd=7168,
             layout="masked", cap=128, gather=True, tokens=1024, skew=0.0, out="bf16"),
        # Prefill of 8 x 4096 tokens, one GPU's share of the first product.
        dict(name="experts prefill", op="matmul", rows=32768, E=32, Nc=4096, Kd=7168,
             layout="contig", cap=0, gather=True, tokens=32768, skew=0.0, out="bf16"),
        # The second product of a 128-expert layer whose experts' popularity falls off steeply:
        # some experts get thousands of rows, some none.
        dict(name="experts skewed", op="matmul", rows=16384, E=128, Nc=2880, Kd=1440,
             layout="contig", cap=0, gather=False, tokens=0, skew=1.2, out="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        c = _draw(rng)
        if 3072 in c.values():
            continue
        w = work(dict(c))
        if c["op"] == "matmul":
            blocks = 0 if c["layout"] == "masked" else _blocks(c["rows"], c["E"])[1]
            if w["flops"] > 1.9e15 or c["E"] * c["Nc"] * c["Kd"] > 9.4e8 \
                    or blocks * c["Nc"] * c["Kd"] > 8.5e9:
                continue
        return c


def _draw(rng):
    op = rng.choice(["gate", "gate_grad", "quant", "matmul"])
    if op in ("gate", "gate_grad"):
        groups = rng.choice([1, 1, 2, 4, 8, 16]) if op == "gate" else 1
        per = _log_int(rng, 4, 512 // groups)
        E = groups * per
        topk_groups = rng.randint((groups + 1) // 2, groups)
        K = rng.randint(1, min(16, topk_groups * per, E))
        renorm = rng.random() < 0.6
        if op == "gate_grad" and renorm:  # the one weight of K = 1 is constant: no gradient
            K = max(2, K)
        c = dict(op=op, N=_log_int(rng, 1, 32768 * 256 // max(E, 256)), E=E, K=K,
                 score=rng.choice([SIGMOID, SOFTMAX]), renorm=renorm,
                 scale=rng.choice([1.0, 2.5]), dtype=rng.choice(["f32", "bf16"]),
                 masked=rng.choice([0.0, 0.0, 0.1]))
        if op == "gate":
            c.update(bias=rng.random() < 0.5, groups=groups, topk_groups=topk_groups,
                     group_top=rng.choice([1, 2]))
        return c
    if op == "quant":
        cols = 16 * _log_int(rng, 4, 448)
        return dict(op=op, rows=_log_int(rng, 1, min(32768, 134217728 // (2 * cols))), cols=cols,
                    act=rng.choice(["none", "swiglu"]), dtype=rng.choice(["bf16", "bf16", "f32"]))
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


def _make_logits(case, g, n):
    """Router logits: normal, with a popularity of its own for each expert; masked experts (a
    failed rank's, say) hold -inf, and where experts are masked at all every 97th token has none."""
    E, dt = case["E"], _dtype(case["dtype"])
    x = torch.randn((n, E), generator=g, device="cuda") * 1.25
    x = x.to(dt)
    if case["masked"] > 0:
        off = torch.rand((n, E), generator=g, device="cuda") < case["masked"]
        x = x.masked_fill(off, -math.inf)
        x[torch.randint(0, 97, (n,), generator=g, device="cuda") == 0] = -math.inf
    return x


def _undecided(case, logits, bias):
    """Rows whose choice hangs on the last bits of a float32: two different values next to each
    other in the order of the first K + 1 experts (or of the groups) are almost equal."""
    keys, gk, scores = _choice64(case, logits, bias)
    loud = scores.max(-1, keepdim=True).values  # sums of a score and a bias may cancel
    top = torch.sort(keys, -1, descending=True).values[:, :case["K"] + 1]
    sets = [top]
    if gk is not None:
        sets.append(torch.sort(gk, -1, descending=True).values[:, :case["topk_groups"] + 1])
    bad = torch.zeros(logits.shape[0], dtype=torch.bool, device=logits.device)
    for v in sets:
        hi, lo = v[:, :-1], v[:, 1:]
        gap = hi - lo
        near = (lo > -math.inf) & (gap > 0) & \
            (gap < 4e-6 * torch.maximum(torch.maximum(hi.abs(), lo.abs()), loud))
        bad |= near.any(-1)
    return bad


def _prepare_gate(case, g):
    N, E = case["N"], case["E"]
    st = dict(case)
    logits = _make_logits(case, g, N)
    bias = None
    if case.get("bias"):
        bias = torch.randn((E,), generator=g, device="cuda") * 0.05
    if case["op"] == "gate":
        # tokens on such a knife's edge are drawn again, so that the 64-bit definition and any
        # order of float32 operations choose the same experts
        if bias is not None or case["groups"] > 1:
            for _ in range(4):
                again = _undecided(case, logits, bias)
                logits = torch.where(again[:, None], _make_logits(case, g, N), logits)
        st.update(logits=logits, bias=bias)
        if own:
            st["out"] = (torch.empty((N, case["K"]), dtype=torch.int32, device="cuda"),
                         torch.empty((N, case["K"]), dtype=torch.float32, device="cuda"))
        return st
    full = dict(case, bias=False, groups=1, topk_groups=1, group_top=1)
    idx, _ = _gate_plain(dict(full, logits=logits, bias=None))
    st.update(logits=logits, idx=idx,
              d_w=torch.randn((N, case["K"]), generator=g, device="cuda") * 1e-2)
    if own:
        st["d_logits"] = torch.empty_like(logits)
    return st


def _prepare_quant(case, g):
    rows, cols = case["rows"], case["cols"]
    wide = 2 * cols if case["act"] == "swiglu" else cols
    x = torch.randn((rows, wide), generator=g, device="cuda")
    # activations: rows of different loudness, a few loud columns
    x *= 0.5 + torch.rand((rows, 1), generator=g, device="cuda")
    x *= 1.0 + 6.0 * (torch.rand((1, wide), generator=g, device="cuda") < 0.01).float()
    st = dict(case, x=x.to(_dtype(case["dtype"])),
              values=torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda"))
    if own:
        st["out"] = (torch.empty((rows, cols), dtype=torch.int8, device="cuda"),
                     torch.empty((rows,), dtype=torch.float32, device="cuda"))
    return st


def _int8(shape, g):
    """Codes of normally distributed values, largest about 4 sigma."""
    out = torch.empty(shape, dtype=torch.int8, device="cuda")
    flat = out.view(-1)
    step = 1 << 27
    for i in range(0, flat.numel(), step):
        n = min(step, flat.numel() - i)
        r = torch.randn((n,), generator=g, device="cuda") * 32.0
        flat[i:i + n] = r.round_().clamp_(-127, 127).to(torch.int8)
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
    st = dict(case, offs=offs, x=_int8((xr, Kd), g), w=_int8((E, Nc, Kd), g))
    st["xs"] = 0.02 + 0.02 * torch.rand((xr,), generator=g, device="cuda")
    st["ws"] = (0.5 + torch.rand((E, Nc), generator=g, device="cuda")) / (32.0 * math.sqrt(Kd))
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
    if case["op"] in ("gate", "gate_grad"):
        return _prepare_gate(case, g)
    return _prepare_quant(case, g) if case["op"] == "quant" else _prepare_matmul(case, g)


# ---- plain forms ------------------------------------------------------------------------------


def _scores_plain(score, x):
    ok = x > -math.inf
    x = torch.clamp(x, max=F32_MAX)
    if score == SIGMOID:
        return torch.where(ok, 1.0 / (1.0 + torch.exp(-x)), 0.0), ok, x
    m = torch.where(ok, x, -math.inf).amax(-1, keepdim=True)
    e = torch.where(ok, torch.exp(x - m), 0.0)
    return e / e.sum(-1, keepdim=True).clamp(min=1e-30), ok, x


def _gate_plain(st):
    s, ok, x = _scores_plain(st["score"], st["logits"].float())
    c = s if st["bias"] is None else s + st["bias"]
    key = x if st["bias"] is None else c
    key = torch.where(ok, key, -math.inf)
    G, N, E = st["groups"], key.shape[0], key.shape[1]
    if G > 1:
        if st["group_top"] == 1:
            gk = key.view(N, G, E // G).amax(-1)
        else:
            two = torch.sort(torch.where(ok, c, -math.inf).view(N, G, E // G), -1,
                             descending=True).values[..., :2]
            gk = two[..., 0] + torch.where(two[..., 1] > -math.inf, two[..., 1], 0.0)
        first = torch.sort(gk, dim=-1, descending=True, stable=True).indices[:, :st["topk_groups"]]
        keep = torch.zeros_like(gk, dtype=torch.bool).scatter_(1, first, True)
        key = torch.where(keep[:, :, None].expand(N, G, E // G).reshape(N, E), key, -math.inf)
    key, idx = torch.sort(key, dim=-1, descending=True, stable=True)
    picked = key[:, :st["K"]] > -math.inf
    idx = idx[:, :st["K"]]
    w = torch.where(picked, s.gather(1, idx), 0.0)
    if st["renorm"]:
        total = w.sum(-1, keepdim=True)
        w = torch.where(total > 0, w / total, 0.0)
    return torch.where(picked, idx, -1).to(torch.int32), w * st["scale"]


def _gate_grad_plain(st):
    x = st["logits"].float()
    s, _, x = _scores_plain(st["score"], x)
    at = st["idx"].long()
    picked = at >= 0
    at = at.clamp(min=0)
    g = torch.where(picked, st["d_w"] * st["scale"], 0.0)
    sk = torch.where(picked, s.gather(1, at), 0.0)
    total = sk.sum(-1, keepdim=True)
    if st["renorm"]:
        q = torch.where(total > 0, sk / total, 0.0)
        g = g - (g * q).sum(-1, keepdim=True)
    if st["score"] == SIGMOID:
        e = torch.exp(-x.gather(1, at).abs())
        ds = e / ((1.0 + e) * (1.0 + e))
        g = g * torch.where(picked, ds, 0.0)
        if st["renorm"]:
            g = torch.where(total > 0, g / total, 0.0)
        d = torch.zeros_like(s).scatter_add_(1, at, g)
    elif st["renorm"]:
        d = torch.zeros_like(s).scatter_add_(1, at, g * q)
    else:
        dense = torch.zeros_like(s).scatter_add_(1, at, g)
        d = s * (dense - (g * sk).sum(-1, keepdim=True))
    return d.to(st["logits"].dtype)


def _quant_plain(st):
    v = st["x"].float()
    if st["act"] == "swiglu":
        a, b = v[:, :st["cols"]], v[:, st["cols"]:]
        v = a / (1.0 + torch.exp(-a)) * b
    top = v.abs().amax(-1, keepdim=True)
    scale = torch.where(top > 0, top / 127.0, 1.0)
    inv = torch.where(top > 0, 127.0 / top, 1.0)
    q = torch.clamp(torch.round(v * inv), -127, 127)
    torch.mul(q, scale, out=st["values"])
    return st["values"], scale.view(-1)


def _blocks(rows, E):
    """Rows of one block of the plain product, and how many blocks there can be."""
    if rows <= 64:
        return 1, rows
    return 128, rows // 128 + min(E, rows)


def _matmul_plain(st):
    E, cap, offs, y = st["E"], st["cap"], st["offs"].long(), st["y"]
    counts = offs[1:] - offs[:-1]
    if st["layout"] == "masked":
        slot = torch.arange(cap, device=y.device)
        valid = slot[None, :] < counts[:, None]
        out_row = torch.arange(E, device=y.device)[:, None] * cap + slot[None, :]
        src = offs[:-1, None] + slot[None, :] if st["gather"] else out_row
        w, ws = st["w"].float(), st["ws"]
    else:
        B, nb = _blocks(st["rows"], E)
        ends = torch.cumsum((counts + B - 1) // B, 0)
        b = torch.arange(nb, device=y.device)
        e = torch.searchsorted(ends, b, right=True).clamp(max=E - 1)
        begin = offs[e] + (b - ends[e] + (counts[e] + B - 1) // B) * B
        out_row = begin[:, None] + torch.arange(B, device=y.device)[None, :]
        valid = (out_row < offs[e + 1][:, None]) & (b < ends[-1])[:, None]
        src = out_row
        w, ws = st["w"][e].float(), st["ws"][e]
    if st["gather"]:
        src = st["row_src"].long()[src.clamp(max=st["rows"] - 1)]
    src = torch.where(valid, src, 0)
    acc = torch.bmm(st["x"][src].float(), w.transpose(1, 2))
    acc = acc * st["xs"][src][..., None] * ws[:, None, :]
    # a block's rows past its expert's end go to one more row, which is dropped
    ext = torch.cat([y, y[:1]])
    ext[torch.where(valid, out_row, y.shape[0]).view(-1)] = acc.view(-1, acc.shape[-1]).to(y.dtype)
    return ext[:-1]


# ---- the framework's calls --------------------------------------------------------------------


def _run_own(st):
    import combine_ep_route_topk_gb300 as ep
    op = st["op"]
    if op == "gate":
        idx, w = ep.ep_gate_topk(
            st["logits"], st["K"],
            ep.EP_SCORE_SIGMOID if st["score"] == SIGMOID else ep.EP_SCORE_SOFTMAX,
            bias=st["bias"], groups=st["groups"], topk_groups=st["topk_groups"],
            group_top=st["group_top"], renorm=st["renorm"], scale=st["scale"],
            topk_idx=st["out"][0], topk_w=st["out"][1])
        return idx, w
    if op == "gate_grad":
        return ep.ep_gate_topk_backward(
            st["d_w"], st["logits"], st["idx"],
            ep.EP_SCORE_SIGMOID if st["score"] == SIGMOID else ep.EP_SCORE_SOFTMAX,
            renorm=st["renorm"], scale=st["scale"], d_logits=st["d_logits"])
    if op == "quant":
        q, scales = ep.ep_quantize_rows(
            st["x"], act=ep.EP_ACT_SWIGLU if st["act"] == "swiglu" else ep.EP_ACT_NONE,
            q=st["out"][0], scales=st["out"][1])
        # the codes are compared as the values they stand for
        torch.mul(q, scales[:, None], out=st["values"])
        return st["values"], scales
    masked = st["layout"] == "masked"
    return ep.ep_expert_matmul(
        st["x"], st["xs"], st["w"], st["ws"], st["offs"],
        layout=ep.EP_LAYOUT_MASKED if masked else ep.EP_LAYOUT_CONTIG, cap=st["cap"],
        row_src=st["row_src"], out=st["y"])


def run(state):
    if own:
        return _run_own(state)
    op = state["op"]
    if op == "gate":
        return _gate_plain(state)
    if op == "gate_grad":
        return _gate_grad_plain(state)
    return _quant_plain(state) if op == "quant" else _matmul_plain(state)


# ---- what a pass cannot do without ------------------------------------------------------------


def work(case):
    op = case["op"]
    if op in ("gate", "gate_grad"):
        N, E, K = case["N"], case["E"], case["K"]
        size = 4 if case["dtype"] == "f32" else 2
        if op == "gate":
            return {"bytes": N * E * size + N * K * 8 + (4 * E if case["bias"] else 0),
                    "flops": 4 * N * E}
        # only an unnormalised softmax needs more of the logits than the picks'
        dense = case["score"] == SOFTMAX and not case["renorm"]
        return {"bytes": N * E * size + N * (E if dense else K) * size + N * K * 8,
                "flops": (6 * E if dense else 12 * K) * N}
    if op == "quant":
        rows, cols = case["rows"], case["cols"]
        wide = 2 * cols if case["act"] == "swiglu" else cols
        size = 4 if case["dtype"] == "f32" else 2
        # the codes and scales written, and the values that the codes stand for
        return {"bytes": rows * (wide * size + cols + 4) + rows * cols * 3, "flops": 4 * rows * wide}
    rows, E, Nc, Kd = case["rows"], case["E"], case["Nc"], case["Kd"]
    size = 4 if case["out"] == "f32" else 2
    share = [i ** -case["skew"] for i in range(1, E + 1)]
    total = sum(share)
    used = sum(1.0 - (1.0 - s / total) ** rows for s in share)  # experts that get any row
    if case["layout"] == "masked":
        rows = sum(min(case["cap"], rows * s / total) for s in share)
    xr = min(case["tokens"], rows) if case["gather"] else rows
    return {"bytes": used * Nc * (Kd + 4) + xr * (Kd + 4) + rows * (Nc * size + 4 * case["gather"]),
            "flops": 2.0 * rows * Nc * Kd}


# ---- 64 bits ----------------------------------------------------------------------------------


def _choice64(case, logits, bias):
    """(experts' keys, groups' keys or None, scores) in 64 bits, experts outside the chosen groups
    and experts without a finite key at -inf."""
    x = logits.double().clamp(max=F32_MAX)
    dead = ~(x > -math.inf)
    if case["score"] == SIGMOID:
        s = torch.sigmoid(x)
    else:
        s = torch.softmax(x.masked_fill(dead, -math.inf), -1)
    s = torch.nan_to_num(s, nan=0.0).masked_fill(dead, 0.0)
    with_bias = s + bias.double() if bias is not None else s
    keys = (with_bias if bias is not None else x).masked_fill(dead, -math.inf)
    if case["groups"] == 1:
        return keys, None, s
    n, G = keys.shape[0], case["groups"]
    shaped = keys.view(n, G, -1)
    if case["group_top"] == 1:
        gk = shaped.max(-1).values
    else:
        v = with_bias.masked_fill(dead, -math.inf).view(n, G, -1).topk(2, -1).values
        gk = v[..., 0] + v[..., 1].masked_fill(v[..., 1] == -math.inf, 0.0)
    # the rank of each group by counting the groups that come before it
    a, b = gk[:, :, None], gk[:, None, :]
    order = torch.arange(G, device=gk.device)
    before = (b > a) | ((b == a) & (order[None, None, :] < order[None, :, None]))
    kept = before.sum(-1) < case["topk_groups"]
    keys = shaped.masked_fill(~kept[:, :, None], -math.inf).reshape(n, -1)
    return keys, gk, s


def _exact_gate(case, seed):
    st = prepare(case, seed)
    keys, _, s = _choice64(case, st["logits"], st["bias"])
    order = torch.argsort(keys, dim=-1, descending=True, stable=True)[:, :case["K"]]
    there = torch.gather(keys, 1, order) != -math.inf
    w = torch.gather(s, 1, order) * there
    if case["renorm"]:
        w = torch.nan_to_num(w / w.sum(-1, keepdim=True), nan=0.0)
    return order.masked_fill(~there, -1).to(torch.int32), w * case["scale"]


def _exact_gate_grad(case, seed):
    st = prepare(case, seed)
    x = st["logits"].double().clamp(max=F32_MAX)
    dead = ~(x > -math.inf)
    s = torch.sigmoid(x) if case["score"] == SIGMOID \
        else torch.softmax(x.masked_fill(dead, -math.inf), -1)
    s = torch.nan_to_num(s, nan=0.0).masked_fill(dead, 0.0)
    # column e of `hit` holds the upstream gradient of expert e's weight, or 0 (not picked)
    up = torch.zeros((x.shape[0], case["E"] + 1), dtype=torch.float64, device="cuda")
    hit = up.scatter(1, st["idx"].long() % (case["E"] + 1), case["scale"] * st["d_w"].double())
    mask = up.scatter(1, st["idx"].long() % (case["E"] + 1), 1.0)[:, :-1]
    hit, picked = hit[:, :-1], s * mask
    if case["renorm"]:
        total = picked.sum(-1, keepdim=True)
        total = total.masked_fill(total == 0, 1.0)
        picked = picked / total
        hit = (hit - (hit * picked).sum(-1, keepdim=True)) * mask
        if case["score"] == SOFTMAX:
            return hit * picked
        return hit / total * s * torch.sigmoid(-x).masked_fill(dead, 0.0)
    if case["score"] == SIGMOID:
        return hit * s * torch.sigmoid(-x).masked_fill(dead, 0.0)
    return s * (hit - (hit * s).sum(-1, keepdim=True))


def _exact_quant(case, seed):
    v = prepare(case, seed)["x"].double()
    if case["act"] == "swiglu":
        v = v[:, :case["cols"]] * torch.sigmoid(v[:, :case["cols"]]) * v[:, case["cols"]:]
    top = v.abs().max(-1, keepdim=True).values
    step = (top / 127).masked_fill(top == 0, 1.0)
    return (v / step).round() * step, step.view(-1)


def _exact_matmul(case, seed):
    """Sums of 1024 products of 8-bit numbers stay below 2^24, where float32 holds every integer:
    each piece of 1024 terms is exact in any order, and the pieces are added in 64 bits."""
    st = prepare(case, seed)
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
        acc = 0.0
        for k in range(0, case["Kd"], 1024):
            piece = st["x"][at, k:k + 1024].float() @ st["w"][e, :, k:k + 1024].float().T
            acc = acc + piece.double()
        out[to:to + hi - lo] = acc * st["xs"][at].double()[:, None] * st["ws"][e].double()[None, :]
    return out


def exact(case, seed):
    op = case["op"]
    if op == "gate":
        return _exact_gate(case, seed)
    if op == "gate_grad":
        return _exact_gate_grad(case, seed)
    return _exact_quant(case, seed) if op == "quant" else _exact_matmul(case, seed)
