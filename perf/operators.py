"""Cases and plain forms of the operators around the head.

Final norm with an 8-bit checkpoint, 8-bit quantisation, the blocked 8-bit
product and row sampling.  ``run`` computes a case in elementary torch
operations, or, with ``own`` set, through the library's entry points.
"""

import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -90  # least group maximum that a scale is made from
GROUP = 128


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def listed():
    return [
        # one decoded token: the norm feeds the 8-bit product directly
        dict(name="norm_fwd token", op="norm_fwd", M=1, D=2048, x="bf16", w="bf16", out="fp8"),
        # a preference pair's rows in training: bf16 head input and checkpoint
        dict(name="norm_fwd pair", op="norm_fwd", M=8192, D=2048, x="bf16", w="f32", out="train"),
        # a short pair with an odd number of rows, fp32 residual stream
        dict(name="norm_bwd odd rows", op="norm_bwd", M=1021, D=1536, x="f32", w="f32", dh="f32"),
        # the long-context pair: gradient from the head's fp32 dH
        dict(name="norm_bwd long", op="norm_bwd", M=32768, D=4096, x="bf16", w="bf16", dh="f32"),
        # activations of a decode batch that come in bf16
        dict(name="quant rows", op="quant", kind="rows", M=250, D=4096, x="bf16"),
        # a head's weights at load time
        dict(name="quant blocks", op="quant", kind="blocks", M=73440, D=1536, x="bf16"),
        # logits of one token: the head is streamed once
        dict(name="product token", op="product", M=1, N=128256, K=4096, c="bf16"),
        # logits of a decode batch of odd size, kept in fp32 for the sampler
        dict(name="product batch", op="product", M=61, N=73440, K=1536, c="f32"),
        # scoring many rows at once
        dict(name="product rows", op="product", M=2048, N=128256, K=4096, c="bf16"),
        # one request, nucleus and top-k
        dict(name="sample one", op="sample", B=1, V=73440, x="f32", k=50, p=0.95, minp=0.0,
             masked=0.0, spread=2.5),
        # a batch with every request's own settings and part of the vocabulary masked
        dict(name="sample mixed", op="sample", B=61, V=128256, x="f32", k=-1, p=-1.0, minp=-1.0,
             masked=0.3, spread=2.5),
        # the largest batch, nucleus alone, bf16 logits full of ties
        dict(name="sample batch", op="sample", B=256, V=262144, x="bf16", k=0, p=0.95, minp=0.0,
             masked=0.0, spread=2.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "quant", "product", "product", "sample", "sample"])
    if op == "norm_fwd":
        return dict(op=op, M=_log(rng, 1, 8192), D=8 * _log(rng, 8, 512),
                    x=rng.choice(["bf16", "f32"]), w=rng.choice(["bf16", "f32"]),
                    out=rng.choice(["fp8", "train", "bf16"]))
    if op == "norm_bwd":
        return dict(op=op, M=_log(rng, 1, 32768), D=8 * _log(rng, 8, 512),
                    x=rng.choice(["bf16", "f32"]), w=rng.choice(["bf16", "f32"]),
                    dh=rng.choice(["bf16", "f32"]))
    if op == "quant":
        kind = rng.choice(["rows", "blocks"])
        return dict(op=op, kind=kind, M=_log(rng, 1, 16384), D=8 * _log(rng, 8, 512),
                    x=rng.choice(["bf16", "f32"]))
    if op == "product":
        return dict(op=op, M=_log(rng, 1, 2048), N=_log(rng, 100, 128256),
                    K=_log(rng, 64, 4096), c=rng.choice(["bf16", "f32"]))
    return dict(op=op, B=_log(rng, 1, 256), V=_log(rng, 1000, 262144),
                x=rng.choice(["bf16", "f32"]), k=rng.choice([0, 1, 50, -1]),
                p=rng.choice([1.0, 0.9, 0.95, -1.0]), minp=rng.choice([0.0, 0.05, -1.0]),
                masked=rng.choice([0.0, 0.3, 0.99]), spread=rng.choice([1.0, 2.5, 4.0]))


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

_T = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _groups(n):
    return -(-n // GROUP)


def _ld(n):
    """Row stride of an 8-bit matrix: whole 16-byte pieces."""
    return -(-n // 16) * 16


def _q_empty(rows, cols):
    return torch.zeros(rows, _ld(cols), dtype=torch.float8_e4m3fn, device="cuda")[:, :cols]


def _f32(*shape):
    return torch.empty(*shape, dtype=torch.float32, device="cuda")


def _residual(g, M, D, dtype):
    """Residual-stream rows: unequal row norms and a few outlying columns."""
    x = _randn(g, M, D) * torch.exp(0.5 * _randn(g, M, 1))
    x[:, torch.randint(0, D, (max(1, D // 256),), generator=g, device="cuda")] *= 20.0
    return x.to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    c, op = case, case["op"]
    s = dict(case=case, ws=torch.zeros(1 << 24, dtype=torch.uint8, device="cuda"))
    if op in ("norm_fwd", "norm_bwd"):
        M, D = c["M"], c["D"]
        x = _residual(g, M, D, _T[c["x"]])
        s["w"] = (1.0 + 0.2 * _randn(g, D)).to(_T[c["w"]])
        s["eps"] = 1e-6
        G = _groups(D)
        if op == "norm_fwd":
            s["x"] = x
            if c["out"] == "fp8":
                s["h8"], s["hs"] = _q_empty(M, D), _f32(M, G)
            else:
                s["h"] = torch.empty(M, D, dtype=torch.bfloat16, device="cuda")
            if c["out"] == "train":
                s["x8"], s["xs"], s["rstd"] = _q_empty(M, D), _f32(M, G), _f32(M)
        else:
            s["rstd"] = torch.rsqrt(x.float().square().mean(1) + s["eps"])
            q, s["xs"] = _quant_rows(x)
            s["x8"] = _q_empty(M, D)
            s["x8"].copy_(q)
            s["dh"] = (_randn(g, M, D) * torch.exp(_randn(g, M, 1)) * 1e-3).to(_T[c["dh"]])
            s["dx"] = torch.empty(M, D, dtype=_T[c["x"]], device="cuda")
            s["dw"] = _f32(D)
    elif op == "quant":
        M, D = c["M"], c["D"]
        s["x"] = (_residual(g, M, D, _T[c["x"]]) if c["kind"] == "rows"
                  else (_randn(g, M, D) * 0.02).to(_T[c["x"]]))
        s["q"] = _q_empty(M, D)
        s["s"] = _f32(M if c["kind"] == "rows" else _groups(M), _groups(D))
    elif op == "product":
        M, N, K = c["M"], c["N"], c["K"]
        a, b = _q_empty(M, K), _q_empty(N, K)
        q, s["sa"] = _quant_rows(_randn(g, M, K))
        a.copy_(q)
        for r in range(0, N, 16384):  # in pieces: only the 8-bit weights are kept
            q, sb = _quant_blocks(_randn(g, min(16384, N - r), K) * 0.02)
            b[r:r + 16384].copy_(q)
            s.setdefault("sb", []).append(sb)
        s["sb"] = torch.cat(s["sb"])
        s["a"], s["b"] = a, b
        s["c"] = torch.empty(M, N, dtype=_T[c["c"]], device="cuda")
    else:
        B, V = c["B"], c["V"]
        # a body of unlikely tokens and some likely ones: from rows that are
        # nearly certain to rows whose mass lies in the body
        l = c["spread"] * _randn(g, B, V)
        hot = torch.randint(0, V, (B, min(64, V // 4)), generator=g, device="cuda")
        sure = 0.2 + torch.rand(B, 1, generator=g, device="cuda")
        e = -torch.log1p(-torch.rand(hot.shape, generator=g, device="cuda"))
        l.scatter_reduce_(1, hot, c["spread"] * (4.0 + 1.5 * sure * e), "amax")
        if c["masked"] > 0:
            l[torch.rand(B, V, generator=g, device="cuda") < c["masked"]] = -math.inf
        if B > 8 and c["masked"] > 0:
            l[B // 2] = -math.inf  # a row that its grammar leaves nothing of
        s["logits"] = l.to(_T[c["x"]])

        def per_row(v, choices, dtype):
            pick = torch.tensor(choices, dtype=dtype, device="cuda")
            at = torch.randint(0, len(choices), (B,), generator=g, device="cuda")
            return pick[at] if v < 0 else torch.full((B,), v, dtype=dtype, device="cuda")

        s["t"] = per_row(-1, [0.0, 0.6, 0.8, 1.0, 1.0, 1.3], torch.float32)
        if c["k"] == 0 and B > 1:
            s["t"].clamp_(min=0.6)
        s["k"] = per_row(c["k"], [0, 20, 50, 200], torch.int32)
        s["p"] = per_row(c["p"], [1.0, 0.8, 0.9, 0.95], torch.float32)
        s["minp"] = per_row(c["minp"], [0.0, 0.0, 0.02, 0.1], torch.float32)
        s["u"] = torch.rand(B, generator=g, device="cuda")
        s["tok"] = torch.empty(B, dtype=torch.int32, device="cuda")
        s["logp"] = _f32(B)
    return s


# --------------------------------------------------------------------------
# plain forms
# --------------------------------------------------------------------------

def _pad(x, rows, cols):
    return torch.nn.functional.pad(x, (0, cols - x.shape[1], 0, rows - x.shape[0]))


def _quant(xg, dims):
    """e4m3 codes of blocks (reduced over ``dims``) and the blocks' scales."""
    m = xg.abs().amax(dims, keepdim=True).clamp(min=TINY)
    return (xg * (E4M3_MAX / m)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), m / E4M3_MAX


def _quant_rows(x):
    M, D = x.shape
    G = _groups(D)
    q, s = _quant(_pad(x.float(), M, G * GROUP).view(M, G, GROUP), (2,))
    return q.view(M, G * GROUP)[:, :D], s.view(M, G)


def _quant_blocks(x):
    N, K = x.shape
    R, G = _groups(N), _groups(K)
    xg = _pad(x.float(), R * GROUP, G * GROUP).view(R, GROUP, G, GROUP)
    q, s = _quant(xg, (1, 3))
    return q.view(R * GROUP, G * GROUP)[:N, :K], s.view(R, G)


def _rows_values(q, s, dtype=torch.float32):
    return q.to(dtype) * s.to(dtype).repeat_interleave(GROUP, 1)[:, :q.shape[1]]


def _blocks_values(q, s, dtype=torch.float32):
    big = s.to(dtype).repeat_interleave(GROUP, 1)[:, :q.shape[1]]
    return q.to(dtype) * big.repeat_interleave(GROUP, 0)[:q.shape[0]]


def _plain_norm_fwd(s):
    x = s["x"].float()
    rstd = torch.rsqrt(x.square().mean(1) + s["eps"])
    h = x * rstd[:, None] * s["w"].float()
    if s["case"]["out"] == "fp8":
        return _quant_rows(h)
    if s["case"]["out"] == "bf16":
        return h.bfloat16()
    return (h.bfloat16(),) + _quant_rows(s["x"]) + (rstd,)


def _plain_norm_bwd(s):
    n = _rows_values(s["x8"], s["xs"]) * s["rstd"][:, None]
    dh = s["dh"].float()
    gw = dh * s["w"].float()
    dx = s["rstd"][:, None] * (gw - n * (gw * n).mean(1, keepdim=True))
    return dx.to(s["dx"].dtype), (dh * n).sum(0)


def _plain_product(s):
    a, b = _rows_values(s["a"], s["sa"]), _blocks_values(s["b"], s["sb"])
    return (a @ b.T).to(s["c"].dtype)


def _plain_sample(s):
    l = s["logits"].double()
    l = torch.where(torch.isnan(l), -math.inf, l)
    B, V = l.shape
    val, idx = torch.sort(l, dim=1, descending=True, stable=True)
    top = val[:, :1]
    t = s["t"].double()[:, None]
    d = torch.where(val == top, 0.0, val - top)  # infinities against infinities too
    live = val > -math.inf
    rank = torch.arange(V, device=l.device)
    w = torch.where(live, torch.exp(d / torch.where(t > 0, t, 1.0)), 0.0)
    k = torch.where(s["k"] > 0, s["k"], V)
    k = torch.where(s["t"] > 0, k, 1)
    w = w * (rank < k[:, None])
    c = torch.cumsum(w, 1)
    p = s["p"].double()[:, None]
    before = torch.cat([torch.zeros_like(top), c[:, :-1]], 1)
    keep = (p >= 1) | (before < p * c[:, -1:]) | (rank == 0)
    keep &= w >= s["minp"].double()[:, None]
    c = torch.cumsum(w * keep, 1)  # down the ranks
    at = (c <= s["u"].double()[:, None] * c[:, -1:]).sum(1, keepdim=True)
    tok = idx.gather(1, at.clamp(max=V - 1))[:, 0]
    empty = ~live[:, 0]
    tok = torch.where(empty, -1, tok)
    lse = torch.exp(torch.where(l == top, 0.0, l - top)).sum(1).log()
    at = l.gather(1, tok.clamp(min=0)[:, None])[:, 0]
    got = torch.where(at == top[:, 0], 0.0, at - top[:, 0]) - lse
    return tok.int(), torch.where(empty, 0.0, got).float()


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------

def _run_own(s):
    from lm_head_cross_flash_b200 import cce
    op = s["case"]["op"]
    if op == "norm_fwd":
        out = s["case"]["out"]
        if out == "fp8":
            cce.cce_norm_forward(s["x"], s["w"], s["eps"], H8=s["h8"], Hs=s["hs"])
            return s["h8"], s["hs"]
        if out == "bf16":
            cce.cce_norm_forward(s["x"], s["w"], s["eps"], H=s["h"])
            return s["h"]
        cce.cce_norm_forward(s["x"], s["w"], s["eps"], H=s["h"], X8=s["x8"], Xs=s["xs"],
                             rstd=s["rstd"])
        return s["h"], s["x8"], s["xs"], s["rstd"]
    if op == "norm_bwd":
        cce.cce_norm_backward(s["x8"], s["xs"], s["rstd"], s["w"], s["dh"], s["dx"], s["dw"],
                              s["ws"])
        return s["dx"], s["dw"]
    if op == "quant":
        f = cce.cce_fp8_quant_rows if s["case"]["kind"] == "rows" else cce.cce_fp8_quant_blocks
        f(s["x"], s["q"], s["s"])
        return s["q"], s["s"]
    if op == "product":
        cce.cce_fp8_matmul(s["a"], s["sa"], s["b"], s["sb"], s["c"], s["ws"])
        return s["c"]
    cce.cce_sample_rows(s["logits"], s["t"], s["k"], s["p"], s["minp"], s["u"], s["tok"],
                        s["logp"])
    return s["tok"], s["logp"]


def run(state):
    if own:
        return _run_own(state)
    op = state["case"]["op"]
    if op == "norm_fwd":
        return _plain_norm_fwd(state)
    if op == "norm_bwd":
        return _plain_norm_bwd(state)
    if op == "quant":
        f = _quant_rows if state["case"]["kind"] == "rows" else _quant_blocks
        return f(state["x"])
    if op == "product":
        return _plain_product(state)
    return _plain_sample(state)


def work(case):
    c, op = case, case["op"]
    size = {"bf16": 2, "f32": 4}
    if op in ("norm_fwd", "norm_bwd"):
        n, rows = c["M"] * c["D"], c["M"] * _groups(c["D"])
        w = c["D"] * size[c["w"]]
        if op == "norm_fwd":
            out = {"fp8": n + 4 * rows, "bf16": 2 * n, "train": 3 * n + 4 * rows + 4 * c["M"]}
            return {"bytes": n * size[c["x"]] + w + out[c["out"]], "flops": 4 * n}
        return {"bytes": n * (1 + size[c["dh"]] + size[c["x"]]) + 4 * rows + 4 * c["M"] + w
                + 4 * c["D"], "flops": 9 * n}
    if op == "quant":
        n = c["M"] * c["D"]
        r = c["M"] if c["kind"] == "rows" else _groups(c["M"])
        return {"bytes": n * (size[c["x"]] + 1) + 4 * r * _groups(c["D"]), "flops": 2 * n}
    if op == "product":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": (M + N) * K + 4 * (M + _groups(N)) * _groups(K)
                + M * N * size[c["c"]], "flops": 2 * M * N * K}
    n = c["B"] * c["V"]
    return {"bytes": n * size[c["x"]] + 28 * c["B"], "flops": 6 * n}


# --------------------------------------------------------------------------
# 64 bits
# --------------------------------------------------------------------------

def _each_group(x):
    """[rows, groups, 128] view of the columns, zeros behind the last."""
    out = x.new_zeros(x.shape[0], _groups(x.shape[1]) * GROUP)
    out[:, :x.shape[1]] = x
    return out.unflatten(1, (-1, GROUP))


def _exact_codes(x, largest):
    """The e4m3 values nearest to 448 x / largest, by their spacing."""
    v = (x * (E4M3_MAX / largest)).double()
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(v / step) * step


def _exact_quant_rows(x):
    xg = _each_group(x)
    big = xg.abs().amax(2, keepdim=True).clamp(min=TINY)
    return _exact_codes(xg, big).flatten(1)[:, :x.shape[1]], (big.double() / E4M3_MAX)[..., 0]


def exact(case, seed):
    s = prepare(case, seed)
    c, op = case, case["op"]
    if op == "norm_fwd":
        x, w = s["x"].double(), s["w"].double()
        r = (x.pow(2).sum(1) / c["D"] + s["eps"]).pow(-0.5)
        h = x * r.unsqueeze(1) * w
        if c["out"] == "bf16":
            return h
        if c["out"] == "fp8":
            return _exact_quant_rows(h)
        return (h,) + _exact_quant_rows(s["x"].float()) + (r,)
    if op == "norm_bwd":
        n = _each_group(s["x8"].double()) * s["xs"].double().unsqueeze(2)
        n = n.flatten(1)[:, :c["D"]] * s["rstd"].double().unsqueeze(1)
        dh = s["dh"].double()
        dn = dh * s["w"].double()
        dot = torch.einsum("md,md->m", dn, n) / c["D"]
        dx = (dn - dot.unsqueeze(1) * n) * s["rstd"].double().unsqueeze(1)
        return dx, torch.einsum("md,md->d", dh, n)
    if op == "quant":
        x = s["x"].float()
        if c["kind"] == "rows":
            return _exact_quant_rows(x)
        R, G = _groups(c["M"]), _groups(c["D"])
        big = x.new_zeros(R * GROUP, G)
        big[:c["M"]] = _each_group(x).abs().amax(2)
        big = big.unflatten(0, (R, GROUP)).amax(1).clamp(min=TINY)
        every = big.repeat_interleave(GROUP, 0)[:c["M"]].repeat_interleave(GROUP, 1)[:, :c["D"]]
        return _exact_codes(x, every), big.double() / E4M3_MAX
    if op == "product":
        M, N, K = c["M"], c["N"], c["K"]
        out = torch.zeros(M, N, dtype=torch.float64, device="cuda")
        rows = torch.arange(N, device="cuda") // GROUP
        for k in range(_groups(K)):  # one block of the inner dimension at a time
            cut = slice(k * GROUP, min(K, (k + 1) * GROUP))
            a = s["a"][:, cut].double() * s["sa"][:, k:k + 1].double()
            b = s["b"][:, cut].double() * s["sb"][rows, k].double().unsqueeze(1)
            out.addmm_(a, b.t())
        return out
    toks, logps = [], []
    for r in range(c["B"]):
        l = s["logits"][r].double()
        l = l.masked_fill(l.isnan(), -math.inf)
        ids = torch.nonzero(l > -math.inf)[:, 0]
        if ids.numel() == 0:
            toks.append(-1)
            logps.append(0.0)
            continue
        l = l[ids]
        d = l - l.max()
        T = float(s["t"][r])
        order = torch.argsort(d, descending=True, stable=True)
        k = 1 if T <= 0 else int(s["k"][r])
        if k > 0:
            order = order[:k]
        w = torch.exp(d[order] / (T if T > 0 else 1.0))
        p = float(s["p"][r])
        n = w.numel()
        if p < 1:
            n = max(1, int((torch.cumsum(w, 0) < p * w.sum()).sum()) + 1)
        n = min(n, max(1, int((w >= float(s["minp"][r])).sum())))
        cum = torch.cumsum(w[:n], 0)
        at = order[min(n - 1, int((cum <= float(s["u"][r]) * cum[-1]).sum()))]
        toks.append(int(ids[at]))
        logps.append(float(d[at] - torch.logsumexp(d, 0)))
    return (torch.tensor(toks, dtype=torch.int32), torch.tensor(logps, dtype=torch.float64))
