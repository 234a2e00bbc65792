"""The unquantized products of a feed-forward layer as measured cases.

Three operators.  The gated block: gate and up projection of each row with its
segment's weights, the activation and the product (forward, optionally keeping
the pre-activations; backward, from the gradient of the block's output through
the down projection to the gradient of the pre-activations, with the activation
formed again).  The segments' linear layer: rows times their segment's weights
(forward, gradient of the rows, gradient of the weights).  Low-rank adapters:
each token's own pair of factors, added to a projection that all tokens share.

Rows and weights are bf16; rows of a segment (an expert, or one segment for a
dense layer) are contiguous, with or without padding between segments.

``run`` computes a case in plain torch operations, or, with ``own`` set, through
the framework's calls.  ``exact`` computes it in 64 bits from the definition.
"""

import math

import torch

own = False

DEV = "cuda"
ALIGN = 128                      # what segments are padded to where they are padded
DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16}


# ----------------------------------------------------------------- the cases

def _gated(M, G, I, K, h, padded=False):
    return dict(op="gated", M=M, G=G, I=I, K=K, h=h, padded=padded)


def _gated_bwd(M, G, I, K, a, padded=False):
    return dict(op="gated_bwd", M=M, G=G, I=I, K=K, a=a, padded=padded)


def _linear(op, M, G, N, K, out, padded=False):
    return dict(op=op, M=M, G=G, N=N, K=K, out=out, padded=padded)


def _lora(T, L, r, N, K, out, runs, none=0.0):
    return dict(op="lora", T=T, L=L, r=r, N=N, K=K, out=out, runs=runs, none=none)


def listed():
    return [
        # one token of a generation step through a dense (shared) block
        dict(_gated(1, 1, 2048, 7168, False), name="gated 1 token"),
        # 16 tokens in flight, 8 experts each, 32 experts here
        dict(_gated(128, 32, 2048, 7168, False), name="gated 16 tokens"),
        # a prefill in training: the experts' rows padded to whole tiles, pre-activations kept
        dict(_gated(8192, 32, 2048, 7168, True, True), name="gated prefill"),
        # training, two experts of eight for 4096 tokens: back through the down projection
        dict(_gated_bwd(8192, 8, 7168, 4096, True), name="gated backward"),
        # a ragged batch with odd widths
        dict(_gated_bwd(1111, 5, 1000, 1992, False, True), name="gated backward odd"),
        # the down projection of the prefill
        dict(_linear("linear", 8192, 32, 7168, 2048, "bf16", True), name="linear prefill"),
        # a short ragged batch, output kept in fp32
        dict(_linear("linear", 515, 6, 1000, 2056, "fp32"), name="linear odd"),
        # gradient of the rows through gate and up
        dict(_linear("linear_dx", 8192, 8, 14336, 4096, "bf16"), name="linear rows' gradient"),
        # gradient of the gate and up weights, kept in fp32
        dict(_linear("linear_dw", 8192, 8, 14336, 4096, "fp32"), name="linear weights' gradient"),
        # a long batch through a small dense layer: few results, long sums
        dict(_linear("linear_dw", 30000, 1, 1024, 1160, "bf16"), name="linear weights' gradient long"),
        # 16 tokens of 16 requests, an adapter each
        dict(_lora(16, 16, 16, 4096, 7168, "bf16", False), name="adapters 16 tokens"),
        # prompts of requests with one of 8 adapters or none, one after the other
        dict(_lora(8192, 8, 64, 4096, 4096, "bf16", True, 0.1), name="adapters prompts"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(("gated", "gated", "gated_bwd", "linear", "linear_dx", "linear_dw", "lora", "lora"))
    out = rng.choice(("fp32", "bf16"))
    flag, padded = rng.random() < 0.5, rng.random() < 0.5
    if kind == "lora":
        runs = rng.random() < 0.5
        T = _log(rng, 16, 8192) if runs else _log(rng, 1, 256)
        r = rng.choice((8, 16, 16, 32, 64, 128))
        L = _log(rng, 1, max(1, min(64, 1024 // r)))
        return _lora(T, L, r, _log(rng, 8, 900) * 8, _log(rng, 8, 900) * 8, out, runs, rng.choice((0.0, 0.1)))
    G = rng.choice((1, 1, _log(rng, 2, 32)))
    M = _log(rng, 1, 16384) if kind in ("gated", "linear") else _log(rng, 64, 32768)
    width, K = _log(rng, 8, 900) * 8, _log(rng, 8, 900) * 8
    # weights of at most 2^28 elements, work below that of the largest listed case
    G = max(1, min(G, (1 << 28) // (2 * width * K)))
    M = max(1, min(M, (1 << 38) // (2 * width * K)))
    padded = padded and G > 1
    if kind == "gated":
        return _gated(M, G, width, K, flag, padded)
    if kind == "gated_bwd":
        return _gated_bwd(M, G, width, K, flag, padded)
    return _linear(kind, M, G, width, K, out, padded)


def _shape(c):
    """Columns that a row brings along the sum, and columns of the product."""
    return (c["I"] * 2 if c["op"] == "gated" else c["I"] if c["op"] == "gated_bwd" else c["N"]), c["K"]


def work(case):
    c = case
    if c["op"] == "lora":
        el = 4 if c["out"] == "fp32" else 2
        T = c["T"] * (1 - c["none"])
        used = c["L"] * (1 - (1 - 1 / c["L"]) ** T) if not c["runs"] else c["L"]
        return {"bytes": used * c["r"] * (c["N"] + c["K"]) * 2 + T * c["K"] * 2 + c["T"] * (2 * c["N"] * el + 4),
                "flops": 2.0 * T * c["r"] * (c["N"] + c["K"])}
    N, K = _shape(c)
    M, G = c["M"], c["G"]
    used = G * (1 - (1 - 1 / G) ** M)                                  # segments with a row
    flops = 2.0 * M * N * K
    if c["op"] == "gated":               # rows and weights in, a (and the pre-activations) out
        return {"bytes": 2 * (M * K + used * N * K + M * c["I"] * (3 if c["h"] else 1)), "flops": flops}
    if c["op"] == "gated_bwd":           # dy, weights, pre-activations in, their gradient (and a) out
        return {"bytes": 2 * (M * K + used * N * K + M * c["I"] * (5 if c["a"] else 4)), "flops": flops}
    el = 4 if c["out"] == "fp32" else 2
    if c["op"] == "linear":
        return {"bytes": 2 * (M * K + used * N * K) + M * N * el, "flops": flops}
    if c["op"] == "linear_dx":
        return {"bytes": 2 * (M * N + used * N * K) + M * K * el, "flops": flops}
    return {"bytes": 2 * M * (N + K) + G * N * K * el, "flops": flops}


# ---------------------------------------------------------------- the inputs

def _segments(c, seed):
    """Rows of each segment (popular experts have more), and where each segment begins and ends."""
    G, M = c["G"], c["M"]
    g = torch.Generator().manual_seed(int(seed))
    popular = torch.exp(0.3 * torch.sin(torch.arange(1, G + 1, dtype=torch.float64)))
    counts = torch.bincount(torch.multinomial(popular, M, replacement=True, generator=g), minlength=G)
    taken = (counts + ALIGN - 1) // ALIGN * ALIGN if c["padded"] else counts
    offsets = torch.zeros(G + 1, dtype=torch.long)
    offsets[1:] = torch.cumsum(taken, 0)
    return counts, offsets


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))

    def randn(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=DEV) * scale).bfloat16()

    if c["op"] == "lora":
        T, L, r, N, K = (c[k] for k in ("T", "L", "r", "N", "K"))
        if c["runs"]:                    # prompts one after the other: up to 2 L runs of tokens
            cuts = torch.sort(torch.randint(0, T, (2 * L - 1,), generator=g, device=DEV)).values
            order = torch.cat([torch.randperm(L, generator=g, device=DEV) for _ in range(2)])
            ids = order[torch.searchsorted(cuts, torch.arange(T, device=DEV), right=True)]
        else:
            ids = torch.randint(0, L, (T,), generator=g, device=DEV)
        if c["none"]:
            share = 16 if c["runs"] else 1
            off = torch.rand((T + share - 1) // share, generator=g, device=DEV) < c["none"]
            ids = torch.where(off.repeat_interleave(share)[:T], torch.full_like(ids, -1), ids)
        return dict(c=c, x=randn(T, K), ids=ids.int(), a=randn(L, r, K, scale=K ** -0.5),
                    b=randn(L, N, r, scale=r ** -0.5), scales=torch.rand(L, generator=g, device=DEV) + 0.5,
                    base=torch.randn(T, N, generator=g, device=DEV).to(DTYPES[c["out"]]))
    counts, offsets = _segments(c, seed)
    G, cap = c["G"], max(int(counts.max()), 1)
    M = c["M"] + (G * (ALIGN - 1) if c["padded"] else 0)     # what padding can come to; rows past the last segment stay
    N, K = _shape(c)
    st = dict(c=c, M=M, offsets=None, counts=None)
    if G > 1:
        st["offsets"] = offsets.int().to(DEV)
        st["counts"] = counts.int().to(DEV) if c["padded"] else None
    # the plain form's plan: rows of each segment side by side, and each row's place among them
    at = torch.arange(cap)[None] + offsets[:-1, None]
    on = torch.arange(cap)[None] < counts[:, None]
    place = torch.full((M + 1,), -1, dtype=torch.long)
    place[torch.where(on, at, torch.full_like(at, M)).reshape(-1)] = torch.arange(G * cap)
    place = place[:M]
    st["at"], st["on"] = at.clamp_max(M - 1).to(DEV), on.to(DEV)
    st["place"], st["live"] = place.clamp_min(0).to(DEV), (place >= 0).to(DEV)[:, None]
    if c["op"] != "linear_dw":
        st["w"] = torch.empty(G, N, K, dtype=torch.bfloat16, device=DEV)
        for e in range(G):
            st["w"][e] = randn(N, K, scale=0.02)
    out = (lambda n, t=torch.bfloat16: torch.zeros(M, n, dtype=t, device=DEV))
    if c["op"] == "gated":               # (rows of padding are left as they are)
        st["x"], st["a"] = randn(M, K), out(c["I"])
        st["h"] = out(N) if c["h"] else None
    elif c["op"] == "gated_bwd":         # the block's [gate | up] pre-activations, and the gradient after the down projection
        st["w"] = st["w"].transpose(1, 2).contiguous()
        st["dy"], st["h"], st["dh"] = randn(M, K), randn(M, 2 * N, scale=1.5), out(2 * N)
        st["a"] = out(N) if c["a"] else None
    elif c["op"] == "linear":
        st["x"], st["y"] = randn(M, K), out(N, DTYPES[c["out"]])
    elif c["op"] == "linear_dx":
        st["dy"], st["dx"] = randn(M, N), out(K, DTYPES[c["out"]])
    else:
        st["dy"], st["x"] = randn(M, N), randn(M, K)
    return st


# ------------------------------------------------------------ the plain forms

def _rows(st, t):
    """[rows, n] to [segments, most rows of one, n] in fp32 (places without a row hold some row)."""
    return t[st["at"]].float()


def _back(st, t, dtype):
    """[segments, most rows of one, n] to [rows, n]; zeros in rows of no segment."""
    rows = t.reshape(-1, t.shape[-1])[st["place"]]
    return torch.where(st["live"], rows, torch.zeros_like(rows)).to(dtype)


def _plain(st):
    c, bf16 = st["c"], torch.bfloat16
    if c["op"] == "lora":
        T, L, r = c["T"], c["L"], c["r"]
        mine = st["ids"].long()[:, None] == torch.arange(L, device=DEV)
        v = torch.matmul(st["x"].float(), st["a"].float().view(L * r, -1).t()).view(T, L, r)
        v = torch.where(mine[..., None], v * st["scales"][:, None], torch.zeros_like(v))
        up = st["b"].float().transpose(1, 2).reshape(L * r, -1)
        return (st["base"].float() + torch.matmul(v.view(T, L * r), up)).to(st["base"].dtype)
    if c["op"] == "gated":
        h = torch.matmul(_rows(st, st["x"]), st["w"].float().transpose(1, 2))
        gate, up = h[..., :c["I"]], h[..., c["I"]:]
        a = _back(st, gate / (1 + torch.exp(-gate)) * up, bf16)
        return (a, _back(st, h, bf16)) if c["h"] else (a,)
    if c["op"] == "gated_bwd":
        da = torch.matmul(_rows(st, st["dy"]), st["w"].float())
        h = _rows(st, st["h"])
        gate, up = h[..., :c["I"]], h[..., c["I"]:]
        s = 1 / (1 + torch.exp(-gate))
        dh = torch.cat((da * up * s * (1 + gate * (1 - s)), da * gate * s), -1)
        dh = _back(st, dh, bf16)
        return (dh, _back(st, gate * s * up, bf16)) if c["a"] else (dh,)
    if c["op"] == "linear":
        return _back(st, torch.matmul(_rows(st, st["x"]), st["w"].float().transpose(1, 2)), DTYPES[c["out"]])
    if c["op"] == "linear_dx":
        return _back(st, torch.matmul(_rows(st, st["dy"]), st["w"].float()), DTYPES[c["out"]])
    dy = _rows(st, st["dy"])
    dy = torch.where(st["on"][..., None], dy, torch.zeros_like(dy))
    return torch.matmul(dy.transpose(1, 2), _rows(st, st["x"])).to(DTYPES[c["out"]])


# ----------------------------------------------------- the framework's own calls

def _own(st):
    import fp4_grouped_gemm_amd as fgg
    c = st["c"]
    if c["op"] == "lora":
        return fgg.lora_add(st["base"], st["x"], st["ids"], st["a"], st["b"], scales=st["scales"])
    seg = dict(offsets=st["offsets"], counts=st["counts"])
    if c["op"] == "gated":
        a, h = fgg.grouped_gated(st["x"], st["w"], **seg, out=st["a"], h=st["h"])
        return (a, h) if c["h"] else (a,)
    if c["op"] == "gated_bwd":
        dh, a = fgg.grouped_gated_backward(st["dy"], st["w"], st["h"], **seg, out=st["dh"], a=st["a"])
        return (dh, a) if c["a"] else (dh,)
    if c["op"] == "linear":
        return fgg.grouped_linear(st["x"], st["w"], **seg, out=st["y"])
    if c["op"] == "linear_dx":
        return fgg.grouped_linear_backward_input(st["dy"], st["w"], **seg, out=st["dx"])
    return fgg.grouped_linear_backward_weight(st["dy"], st["x"], c["G"], **seg, out_dtype=DTYPES[c["out"]])


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------- 64 bits

def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "lora":
        out = st["base"].double()
        for e in range(c["L"]):          # adapter by adapter, its tokens only
            t = torch.nonzero(st["ids"] == e)[:, 0]
            if t.numel():
                v = st["x"][t].double() @ st["a"][e].double().t()
                out[t] += st["scales"][e].double() * (v @ st["b"][e].double().t())
        return out
    counts, offsets = (t.tolist() for t in _segments(c, seed))
    M, (N, K), I = st["M"], _shape(c), c.get("I", 0)
    zeros = (lambda *shape: torch.zeros(*shape, dtype=torch.float64, device=DEV))
    if c["op"] == "gated":
        one, two = zeros(M, I), zeros(M, N) if c["h"] else None
    elif c["op"] == "gated_bwd":
        one, two = zeros(M, 2 * I), zeros(M, I) if c["a"] else None
    elif c["op"] == "linear_dw":
        one, two = zeros(c["G"], N, K), None
    else:
        one, two = zeros(M, N if c["op"] == "linear" else K), None
    for e in range(c["G"]):
        at = slice(offsets[e], offsets[e] + counts[e])
        if counts[e] == 0:
            continue
        if c["op"] == "gated":
            h = st["x"][at].double() @ st["w"][e].double().t()
            one[at] = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
            if c["h"]:
                two[at] = h
        elif c["op"] == "gated_bwd":     # by automatic differentiation of the definition
            h = st["h"][at].double().requires_grad_()
            a = torch.nn.functional.silu(h[:, :I]) * h[:, I:]
            a.backward(st["dy"][at].double() @ st["w"][e].double())
            one[at] = h.grad
            if c["a"]:
                two[at] = a.detach()
        elif c["op"] == "linear":
            one[at] = st["x"][at].double() @ st["w"][e].double().t()
        elif c["op"] == "linear_dx":
            one[at] = st["dy"][at].double() @ st["w"][e].double()
        else:
            one[e] = st["dy"][at].double().t() @ st["x"][at].double()
    if c["op"].startswith("gated"):
        return (one,) if two is None else (one, two)
    return one
