"""The expert-routing operators of a mixture-of-experts layer as measured cases.

Four operators, each in the directions it has: the router (logits to expert ids
and gate weights, and its gradient), tokens sorted into expert order (optionally
scaled by their gate weights, and the gradient), rows brought back to token
order as a weighted sum (and the gradient, the gate weights' included), and the
matrix-vector product of few tokens with 4-bit expert weights (E2M1 codes with
one power-of-two scale per 32 along K; plain, with SiLU(gate)*up, or with the
gate-weighted sum over a token's experts).

``run`` computes a case in plain torch operations, or, with ``own`` set, through
the framework's calls.  ``exact`` computes it in 64 bits from the definition.
"""

import math

import torch

own = False

DEV = "cuda"
ALIGN = 128                      # expert segments are padded to whole GEMM tiles
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


# ----------------------------------------------------------------- the cases

def _route(op, T, E, k, dtype, gate, bias, renorm, masked=0.0):
    return dict(op=op, T=T, E=E, k=k, dtype=dtype, gate=gate, bias=bias, renorm=renorm, masked=masked)


def _rows(op, T, E_all, E, k, N, dtype, weights):
    return dict(op=op, T=T, E_all=E_all, E=E, k=k, N=N, dtype=dtype, weights=weights)


def _gemv(T, G, k, N, K, mode, tiled, out):
    return dict(op="gemv", T=T, G=G, k=k, N=N, K=K, mode=mode, tiled=tiled, out=out)


def listed():
    return [
        # one token of a generation step: sigmoid gate with a balancing bias, 8 of 256 experts
        dict(_route("route", 1, 256, 8, "fp32", "sigmoid", True, True), name="route 1 token"),
        # a prefill of 8192 tokens, bf16 logits (ties are common), renormalized softmax
        dict(_route("route", 8192, 256, 8, "bf16", "softmax", False, True, 0.01), name="route prefill"),
        # the same layer in training: softmax over 160 experts, gradient of every logit
        dict(_route("route_bwd", 16384, 160, 6, "fp32", "softmax", False, False), name="route backward"),
        # prefill on one of 8 GPUs: 32 of 256 experts are local
        dict(_rows("permute", 8192, 256, 32, 8, 7168, "bf16", False), name="permute prefill"),
        # training, two experts of eight per token, all local: gradient of the hidden states
        dict(_rows("permute_bwd", 4096, 8, 8, 2, 4096, "fp32", False), name="permute backward"),
        # a short batch with an odd hidden size
        dict(_rows("unpermute", 515, 64, 64, 6, 1999, "fp32", True), name="unpermute odd"),
        # a few tokens in flight
        dict(_rows("unpermute", 9, 64, 64, 8, 2048, "bf16", True), name="unpermute few"),
        # training: gradients of the experts' outputs and of the gate weights
        dict(_rows("unpermute_bwd", 8192, 32, 32, 4, 4096, "bf16", True), name="unpermute backward"),
        # one token through a dense 4-bit projection
        dict(_gemv(1, 1, 1, 4096, 7168, "plain", True, "bf16"), name="gemv 1 token"),
        # a ragged batch of 13 tokens, weights as quantized, output kept in fp32
        dict(_gemv(13, 1, 1, 7001, 2048, "plain", False, "fp32"), name="gemv 13 tokens"),
        # the gate and up projections of the 8 experts of one token
        dict(_gemv(1, 32, 8, 2048, 7168, "silu", True, "bf16"), name="experts gate-up 1 token"),
        # the down projections of 16 tokens, summed with the gate weights
        dict(_gemv(16, 32, 8, 7168, 2048, "sum", False, "bf16"), name="experts down 16 tokens"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("route", "route_bwd", "permute", "permute_bwd", "unpermute", "unpermute_bwd", "gemv", "gemv"))
    dtype = rng.choice(("fp32", "bf16"))
    if kind in ("route", "route_bwd"):
        E = _log(rng, 4, 384)
        return _route(kind, _log(rng, 1, 16384), E, min(E, rng.randint(1, 10)), dtype,
                      rng.choice(("softmax", "sigmoid")), kind == "route" and rng.random() < 0.5,
                      rng.random() < 0.5, rng.choice((0.0, 0.05)))
    if kind != "gemv":
        E = _log(rng, 2, 64)
        share = rng.choice((1, 1, 4))
        k = min(E, rng.randint(1, 8))
        N = _log(rng, 60, 7200)
        if rng.random() < 0.5:
            N = (N + 63) // 64 * 64
        T = min(_log(rng, 1, 8192), max(1, (1 << 26) // (k * N)))
        return _rows(kind, T, E * share, E, k, N, dtype, rng.random() < 0.5)
    mode = rng.choice(("plain", "silu", "sum"))
    G = 1 if mode == "plain" and rng.random() < 0.5 else _log(rng, 2, 32)
    k = min(G, rng.randint(1, 8))
    tiled = rng.random() < 0.5
    K = _log(rng, 4, 224) * 32
    N = _log(rng, 40, 7200)
    if tiled:
        K, N = (K + 127) // 128 * 128, (N + 15) // 16 * 16
    N = min(N, (1 << 28) // (G * K) // 16 * 16)
    return _gemv(rng.randint(1, 16), G, k, N, K, mode, tiled, rng.choice(("fp32", "bf16")))


def _capacity(c):
    """Rows that the sorted buffer holds: every pair with its padding, or on one of several GPUs a fourth
    more than the local pairs to be expected (what is beyond is dropped)."""
    if c["E"] == c["E_all"]:
        return c["T"] * c["k"] + c["E"] * (ALIGN - 1)
    return c["T"] * c["k"] * c["E"] * 5 // (c["E_all"] * 4) + c["E"] * ALIGN


def work(case):
    c = case
    if c["op"] in ("route", "route_bwd"):
        el = 4 if c["dtype"] == "fp32" else 2
        n, pairs = c["T"] * c["E"], c["T"] * c["k"]
        if c["op"] == "route":
            return {"bytes": n * el + pairs * 8 + (4 * c["E"] if c["bias"] else 0), "flops": 5 * n}
        # only the selected logits matter unless the softmax's normalizer runs over the whole row
        whole = c["gate"] == "softmax" and not c["renorm"]
        return {"bytes": (n if whole else pairs) * el + pairs * 8 + n * el, "flops": (6 if whole else 1) * n}
    if c["op"] != "gemv":
        el = 4 if c["dtype"] == "fp32" else 2
        pairs = c["T"] * c["k"] * c["E"] / c["E_all"]
        held = c["T"] * (1 - (1 - c["E"] / c["E_all"]) ** c["k"])      # tokens with a local expert
        rows = pairs * c["N"] * el
        used = c["E"] * (1 - (1 - 1 / c["E_all"]) ** (c["T"] * c["k"]))   # experts with a row
        padded = used * ALIGN * max(1.0, pairs / used / ALIGN + 0.5) * c["N"] * el
        if c["op"] == "permute":         # tokens in, rows (padding to the segments' end included) out
            total = held * c["N"] * el + padded
        elif c["op"] == "permute_bwd":   # rows in, tokens out; with weights the tokens in too
            total = rows + c["T"] * c["N"] * el + (held * c["N"] * el if c["weights"] else 0)
        elif c["op"] == "unpermute":
            total = rows + c["T"] * c["N"] * el
        else:                            # tokens in, rows out; with weights the rows in too
            total = held * c["N"] * el + padded + (rows if c["weights"] else 0)
        return {"bytes": total + c["T"] * c["k"] * 8, "flops": pairs * c["N"] * (4 if c["weights"] else 1)}
    used = c["G"] * (1 - (1 - c["k"] / c["G"]) ** c["T"])              # distinct experts of T tokens
    width = c["N"] * (2 if c["mode"] == "silu" else 1)
    weights = used * width * (c["K"] / 2 + c["K"] / 32)
    slots = c["T"] * c["k"]
    x = (slots if c["mode"] == "sum" else c["T"]) * c["K"] * 2
    y = (c["T"] if c["mode"] == "sum" else slots) * c["N"] * (4 if c["out"] == "fp32" else 2)
    return {"bytes": weights + x + y, "flops": 2.0 * slots * width * c["K"]}


# ---------------------------------------------------------------- the inputs

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _choose(g, T, E_all, k):
    """Distinct experts of each token, popular ones more often (slots in no particular order)."""
    popular = 0.6 * torch.sin(torch.arange(1, E_all + 1, device=DEV, dtype=torch.float32))
    noise = torch.rand(T, E_all, generator=g, device=DEV).clamp_(1e-9, 1 - 1e-7)
    return torch.topk(popular - torch.log(-torch.log(noise)), k, dim=1).indices.int()


def _maps(ids, E, M):
    """Stable sort of the (token, slot) pairs by expert, segments padded to ALIGN; rows from M on are dropped."""
    flat = ids.reshape(-1).long()
    flat = torch.where((flat >= 0) & (flat < E), flat, torch.full_like(flat, E))
    counts = torch.bincount(flat, minlength=E + 1)[:E]
    padded = (counts + ALIGN - 1) // ALIGN * ALIGN
    offsets = torch.zeros(E + 1, dtype=torch.long, device=DEV)
    offsets[1:] = torch.cumsum(padded, 0)
    order = torch.argsort(flat, stable=True)
    starts = torch.zeros(E + 1, dtype=torch.long, device=DEV)
    starts[1:] = torch.cumsum(counts, 0)
    e = flat[order]
    local = e < E
    rows = offsets[e[local]] + torch.arange(flat.numel(), device=DEV)[local] - starts[e[local]]
    src_to_row = torch.full_like(flat, -1)
    src_to_row[order[local]] = torch.where(rows < M, rows, torch.full_like(rows, -1))
    row_to_src = torch.full((M,), -1, dtype=torch.long, device=DEV)
    row_to_src[rows[rows < M]] = order[local][rows < M]
    return src_to_row.int(), row_to_src.int(), offsets.int()


def _quantize(w):
    """E2M1 codes (two a byte, the even element low) and E8M0 scale bytes, one per 32 along K."""
    n, K = w.shape
    b = w.view(n, K // 32, 32)
    amax = b.abs().amax(-1).clamp_min(1e-30)
    e = torch.ceil(torch.log2(amax / 6.0)).clamp(-127, 127)
    q = b / torch.exp2(e)[..., None]
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=DEV)
    code = torch.bucketize(q.abs(), edges).to(torch.uint8) | ((q < 0).to(torch.uint8) << 3)
    code = code.view(n, K // 2, 2)
    return code[..., 0] | (code[..., 1] << 4), (e + 127).to(torch.uint8)


def _tiles(b, s):
    """16-row x 128-element tiles, 16-byte pieces column by column; scales in 256-byte spans of 16 rows x 16."""
    G, N, Kh = b.shape
    bt = b.view(G, N // 16, 16, Kh // 64, 4, 16).permute(0, 1, 3, 4, 2, 5).contiguous().view(G, -1)
    spans = (s.shape[2] + 15) // 16
    pad = torch.full((G, N, spans * 16), 127, dtype=torch.uint8, device=DEV)
    pad[:, :, :s.shape[2]] = s
    st = pad.view(G, N // 16, 16, spans, 16).permute(0, 1, 3, 2, 4).contiguous().view(G, -1)
    return bt, st


def prepare(case, seed):
    c, g = dict(case), _generator(seed)
    if c["op"] in ("route", "route_bwd"):
        T, E, k = c["T"], c["E"], c["k"]
        logits = torch.randn(T, E, generator=g, device=DEV) * 1.5
        logits += torch.randn(E, generator=g, device=DEV) * 0.5
        if c["masked"]:                  # experts closed to a token, and tokens (padding) without any
            shut = torch.rand(T, E, generator=g, device=DEV) < c["masked"]
            shut |= (torch.rand(T, 1, generator=g, device=DEV) < c["masked"] / 8)
            logits.masked_fill_(shut, -math.inf)
        st = dict(c=c, logits=logits.to(DTYPES[c["dtype"]]).contiguous(), bias=None)
        if c["bias"]:
            st["bias"] = torch.randn(E, generator=g, device=DEV) * 0.05
        if c["op"] == "route_bwd":
            st["ids"] = _plain_route(st["logits"], None, k, c["gate"], c["renorm"])[0]
            st["dw"] = torch.randn(T, k, generator=g, device=DEV)
        return st
    if c["op"] != "gemv":
        T, k, N, dt = c["T"], c["k"], c["N"], DTYPES[c["dtype"]]
        M = _capacity(c)
        s2r, r2s, offsets = _maps(_choose(g, T, c["E_all"], k), c["E"], M)
        st = dict(c=c, s2r=s2r, r2s=r2s, offsets=offsets, w=None)
        if c["weights"]:
            st["w"] = torch.softmax(torch.rand(T, k, generator=g, device=DEV), dim=1)
        if c["op"] in ("permute", "unpermute_bwd"):      # rows past the last segment are left as they are
            st["out"] = torch.zeros(M, N, dtype=dt, device=DEV)
        st["tokens"] = torch.randn(T, N, generator=g, device=DEV).to(dt)
        if c["op"] in ("unpermute", "permute_bwd") or c["weights"]:
            st["rows"] = torch.randn(M, N, generator=g, device=DEV).to(dt)
        return st
    T, G, k, N, K = c["T"], c["G"], c["k"], c["N"], c["K"]
    width = N * (2 if c["mode"] == "silu" else 1)
    b = torch.empty(G, width, K // 2, dtype=torch.uint8, device=DEV)
    s = torch.empty(G, width, K // 32, dtype=torch.uint8, device=DEV)
    for e in range(G):
        b[e], s[e] = _quantize(torch.randn(width, K, generator=g, device=DEV) * 0.02)
    st = dict(c=c, b=b, s=s, ids=None, w=None)
    if c["tiled"]:
        st["bt"], st["st"] = _tiles(b, s)    # the layout in which the weights are kept, made once
    if G > 1:
        st["ids"] = _choose(g, T, G, k)
    if c["mode"] == "sum":
        st["w"] = torch.softmax(torch.rand(T, k, generator=g, device=DEV), dim=1)
        st["x"] = torch.randn(T, k, K, generator=g, device=DEV).bfloat16()
    else:
        st["x"] = torch.randn(T, K, generator=g, device=DEV).bfloat16()
    return st


# ------------------------------------------------------------ the plain forms

def _plain_route(logits, bias, k, gate, renorm, scale=1.0):
    """ids and weights: the k largest of the logits (of score + bias with a bias), ties to the lower
    id; an expert at -inf is never chosen, a slot left over has id -1 and weight 0."""
    x = logits.float()
    if bias is None:
        key = x
    else:                                # score + bias in 64 bits: values next to the k-th
        d = x.double()
        key = (torch.sigmoid(d) if gate == "sigmoid" else _plain_softmax(d)) + bias.double()
    key = torch.where(x > -math.inf, key, torch.full_like(key, -math.inf))
    top, at = torch.sort(key, dim=1, descending=True, stable=True)
    top, at = top[:, :k], at[:, :k]
    on = top > -math.inf
    chosen = torch.gather(x, 1, at)
    if gate == "sigmoid":
        w = torch.where(on, torch.sigmoid(chosen), torch.zeros_like(chosen))
        if renorm:
            w = w / w.sum(1, keepdim=True)
    elif renorm:
        w = _plain_softmax(torch.where(on, chosen, torch.full_like(chosen, -math.inf)))
    else:
        w = torch.gather(_plain_softmax(x), 1, at)
    w = torch.where(on, w * scale, torch.zeros_like(w))
    return torch.where(on, at, torch.full_like(at, -1)).int(), w


def _plain_softmax(x):
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route_bwd(logits, ids, dw, gate, renorm, scale=1.0):
    x, on = logits.float(), ids >= 0
    at = ids.clamp_min(0).long()
    dw = torch.where(on, dw * scale, torch.zeros_like(dw))
    out = torch.zeros_like(x)
    if gate == "softmax" and not renorm:
        s = torch.where(x.amax(1, keepdim=True) > -math.inf, _plain_softmax(x), torch.zeros_like(x))
        out.scatter_add_(1, at, dw)
        out = s * (out - (out * s).sum(1, keepdim=True))
    else:
        chosen = torch.gather(x, 1, at)
        s = torch.where(on, torch.sigmoid(chosen), torch.zeros_like(chosen))
        if renorm:
            if gate == "softmax":
                p = _plain_softmax(torch.where(on, chosen, torch.full_like(chosen, -math.inf)))
                s = torch.zeros_like(p)
            else:
                p = s / s.sum(1, keepdim=True)
            p = torch.where(on, p, torch.zeros_like(p))
            d = p * (1 - s) * (dw - (dw * p).sum(1, keepdim=True))
        else:
            d = dw * s * (1 - s)
        out.scatter_add_(1, at, torch.where(on, d, torch.zeros_like(d)))
    return out.to(logits.dtype)


def _plain_to_rows(tokens, s2r, r2s, w):
    """rows[r] = w[p] * tokens[p // k] for the pair p of row r, zeros for all other rows."""
    k = s2r.numel() // tokens.shape[0]
    p = r2s.long()
    on = p >= 0
    rows = tokens[p.clamp_min(0) // k]
    if w is not None:
        rows = rows.float() * w.reshape(-1)[p.clamp_min(0)][:, None]
    return torch.where(on[:, None], rows, torch.zeros_like(rows)).to(tokens.dtype)


def _plain_to_tokens(rows, s2r, T, w):
    """tokens[t] = sum over the slots j of w[t, j] * rows[row of (t, j)]."""
    r = s2r.view(T, -1).long()
    scale = (r >= 0).float() if w is None else torch.where(r >= 0, w, torch.zeros_like(w))
    picked = rows[r.clamp_min(0).reshape(-1)].float().view(T, r.shape[1], -1)
    return (picked * scale[..., None]).sum(1).to(rows.dtype)


def _plain_dots(tokens, rows, s2r):
    """dw[t, j] = <tokens[t], rows[row of (t, j)]>, 0 where the pair has no row."""
    T = tokens.shape[0]
    r = s2r.view(T, -1).long()
    picked = rows[r.clamp_min(0).reshape(-1)].float().view(T, r.shape[1], -1)
    d = (picked * tokens.float()[:, None]).sum(-1)
    return torch.where(r >= 0, d, torch.zeros_like(d))


def _plain_weights(b, s):
    """[.., K/2] codes and [.., K/32] scale bytes to fp32 values."""
    table = torch.tensor(E2M1, device=b.device)
    v = torch.stack((table[(b & 15).int()], table[(b >> 4).int()]), -1).view(*b.shape[:-1], -1, 32)
    return (v * torch.exp2(s.float() - 127.0)[..., None]).view(*b.shape[:-1], -1)


def _plain_gemv(st):
    c, x = st["c"], st["x"].float()
    T, k, G = c["T"], c["k"], c["G"]
    if st["ids"] is None:                # one set of weights
        y = torch.matmul(x.view(-1, c["K"]), _plain_weights(st["b"][0], st["s"][0]).t()).view(T, k, -1)
    else:
        x = x if x.dim() == 3 else x[:, None].expand(T, k, c["K"])
        ids = st["ids"].long()
        if T * k < G:                    # fewer products than experts: only the chosen experts' weights
            at = ids.reshape(-1)
            y = torch.bmm(_plain_weights(st["b"][at], st["s"][at]), x.reshape(T * k, -1, 1)).view(T, k, -1)
        else:                            # every expert with every pair, then the pair's own
            y = torch.matmul(x.reshape(T * k, -1), _plain_weights(st["b"], st["s"]).transpose(1, 2))
            y = y[ids.reshape(-1), torch.arange(T * k, device=x.device)].view(T, k, -1)
    if c["mode"] == "silu":
        gate, up = y[..., :c["N"]], y[..., c["N"]:]
        y = gate / (1 + torch.exp(-gate)) * up
    if c["mode"] == "sum":
        y = (y * st["w"][..., None]).sum(1)
    elif st["ids"] is None:
        y = y[:, 0]
    return y.to(DTYPES[c["out"]])


def _plain(st):
    c = st["c"]
    if c["op"] == "route":
        return _plain_route(st["logits"], st["bias"], c["k"], c["gate"], c["renorm"])
    if c["op"] == "route_bwd":
        return _plain_route_bwd(st["logits"], st["ids"], st["dw"], c["gate"], c["renorm"])
    if c["op"] == "permute":
        return _plain_to_rows(st["tokens"], st["s2r"], st["r2s"], st["w"])
    if c["op"] == "unpermute":
        return _plain_to_tokens(st["rows"], st["s2r"], c["T"], st["w"])
    if c["op"] == "permute_bwd":         # rows: the gradient that comes in; tokens: the forward's input
        dx = _plain_to_tokens(st["rows"], st["s2r"], c["T"], st["w"])
        return (dx, _plain_dots(st["tokens"], st["rows"], st["s2r"])) if c["weights"] else (dx,)
    if c["op"] == "unpermute_bwd":       # tokens: the gradient that comes in; rows: the forward's input
        dr = _plain_to_rows(st["tokens"], st["s2r"], st["r2s"], st["w"])
        return (dr, _plain_dots(st["tokens"], st["rows"], st["s2r"])) if c["weights"] else (dr,)
    return _plain_gemv(st)


# ----------------------------------------------------- the framework's own calls

def _own(st):
    import fp4_grouped_gemm_amd as fgg
    c = st["c"]
    if c["op"] == "route":
        return fgg.moe_route(st["logits"], c["k"], gate=c["gate"], bias=st["bias"], renormalize=c["renorm"])
    if c["op"] == "route_bwd":
        return fgg.moe_route_backward(st["logits"], st["ids"], st["dw"], gate=c["gate"], renormalize=c["renorm"])
    if c["op"] == "permute":
        return fgg.moe_permute_rows(st["tokens"], st["s2r"], st["r2s"], st["offsets"], topk_w=st["w"],
                                    out=st["out"])
    if c["op"] == "unpermute":
        return fgg.moe_unpermute_rows(st["rows"], st["s2r"], c["T"], topk_w=st["w"])
    if c["op"] == "permute_bwd":
        dx, dw = fgg.moe_permute_rows_backward(st["rows"], st["s2r"], c["T"], topk_w=st["w"],
                                               x=st["tokens"] if c["weights"] else None)
        return (dx, dw) if c["weights"] else (dx,)
    if c["op"] == "unpermute_bwd":
        dr, dw = fgg.moe_unpermute_rows_backward(st["tokens"], st["s2r"], st["r2s"], st["offsets"], topk_w=st["w"],
                                                 rows=st["rows"] if c["weights"] else None, out=st["out"])
        return (dr, dw) if c["weights"] else (dr,)
    b, s, q = ((st["bt"], st["st"], fgg.Q_E2M1_E8M0_1x32_TILED) if c["tiled"] else
               (st["b"], st["s"], fgg.Q_E2M1_E8M0_1x32))
    return fgg.moe_gemv_fp4(st["x"], b, s, topk_ids=st["ids"], topk_w=st["w"], b_qdesc=q, n=c["N"],
                            silu_mul=c["mode"] == "silu", out_dtype=DTYPES[c["out"]])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- 64 bits

def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        x = st["logits"].double()
        p = torch.sigmoid(x) if c["gate"] == "sigmoid" else torch.nan_to_num(torch.softmax(x, 1))
        key = x if st["bias"] is None else torch.where(x == -math.inf, x, p + st["bias"].double())
        ids = torch.empty(T, k, dtype=torch.long, device=DEV)
        left = key.clone()
        for j in range(k):               # the largest that is left, the first of equals
            best = left.amax(1, keepdim=True)
            first = torch.where(left == best, torch.arange(E, device=DEV), E).amin(1)
            ids[:, j] = torch.where(best[:, 0] == -math.inf, -1, first)
            left.scatter_(1, first[:, None], -math.inf)
        w = torch.where(ids < 0, 0.0, torch.gather(p, 1, ids.clamp_min(0)))
        if c["renorm"]:
            w = torch.nan_to_num(w / w.sum(1, keepdim=True))
        return ids.int(), w
    if c["op"] == "route_bwd":           # by automatic differentiation of the definition
        x = st["logits"].double().requires_grad_()
        ids, none = st["ids"].long().clamp_min(0), st["ids"] < 0
        empty = torch.isneginf(x).all(1, keepdim=True)
        safe = torch.where(empty, torch.zeros_like(x), x)
        if c["gate"] == "sigmoid":
            w = torch.gather(torch.sigmoid(safe), 1, ids)
        else:
            w = torch.gather(torch.softmax(safe, 1), 1, ids)
        w = torch.where(none, torch.zeros_like(w), w)
        if c["renorm"]:
            w = w / torch.where(empty, torch.ones_like(w[:, :1]), w.sum(1, keepdim=True))
        w.backward(st["dw"].double())
        return x.grad
    if c["op"] != "gemv":
        T, k, N = c["T"], c["k"], c["N"]
        r = st["s2r"].view(T, k).long()
        w = st["w"].double() if c["weights"] else torch.ones(T, k, dtype=torch.float64, device=DEV)
        tokens = st["tokens"].double()
        dots = torch.zeros(T, k, dtype=torch.float64, device=DEV)
        if c["op"] in ("permute", "unpermute_bwd"):
            out = torch.zeros(st["r2s"].numel(), N, dtype=torch.float64, device=DEV)
        else:
            out = torch.zeros(T, N, dtype=torch.float64, device=DEV)
        for j in range(k):               # slot by slot: the rows of one slot are all different
            t = torch.nonzero(r[:, j] >= 0)[:, 0]
            rj = r[t, j]
            if c["op"] in ("permute", "unpermute_bwd"):
                out[rj] = tokens[t] * w[t, j][:, None]
            else:
                out[t] += st["rows"][rj].double() * w[t, j][:, None]
            if c["weights"] and c["op"].endswith("bwd"):
                dots[t, j] = (tokens[t] * st["rows"][rj].double()).sum(1)
        if c["op"].endswith("bwd"):
            return (out, dots) if c["weights"] else (out,)
        return out
    T, k, N, K = c["T"], c["k"], c["N"], c["K"]
    ids = torch.zeros(T, k, dtype=torch.long, device=DEV) if st["ids"] is None else st["ids"].long()
    x = st["x"].double().view(T, -1, K).expand(T, k, K)
    y = torch.zeros(T, k, st["b"].shape[1], dtype=torch.float64, device=DEV)
    value = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    for e in range(c["G"]):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel() == 0:
            continue
        b = st["b"][e].long()
        v = torch.empty(b.shape[0], K, dtype=torch.float64, device=DEV)
        v[:, 0::2] = value[b % 16]
        v[:, 1::2] = value[b // 16]
        v *= torch.pow(2.0, st["s"][e].double() - 127).repeat_interleave(32, dim=1)
        y[t, j] = x[t, j] @ v.t()
    if c["mode"] == "silu":
        y = torch.nn.functional.silu(y[..., :N]) * y[..., N:]
    if c["mode"] == "sum":
        return (y * st["w"].double()[..., None]).sum(1)
    return y[:, 0] if st["ids"] is None else y
