"""The operators around the head as they are used together: a decoding step
samples tokens, the tokens become labels, and a training pass runs from the
residual stream to its gradient; both also captured into graphs.

Tolerances: what the head itself is held to (log-probs 2e-3 absolute, loss
1e-3 and gradients 1e-2 relative); sampled tokens follow from the logits that
the step itself made, so they are compared for equality.
"""

import numpy as np
import pytest
import torch

from lm_head_cross_flash_b200 import cce
from oracle import flash_cce as F
from oracle import head_ops as O

from helpers import TOL_DH, TOL_LOGP, TOL_LOSS, rel_fro

pytestmark = pytest.mark.gpu

EPS = 1e-6


def make(seed, M, D, V, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda").manual_seed(seed)
    X = (torch.randn(M, D, generator=g, device="cuda") * 3).to(dtype)
    w = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(dtype)
    W = (torch.randn(V, D, generator=g, device="cuda") * 2 / D ** 0.5).to(dtype)
    return X, w, W, torch.rand(M, generator=g, device="cuda")


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def settings(B):
    r = np.random.default_rng(3)
    t = lambda a, d=torch.float32: torch.tensor(a, dtype=d, device="cuda")
    return dict(temperature=t(r.choice([0.0, 0.8, 1.0, 1.2], B)),
                top_k=t(r.choice([0, 20, 200], B), torch.int32), top_p=t(r.choice([1.0, 0.9], B)),
                min_p=t(r.choice([0.0, 0.02], B)))


@pytest.mark.parametrize("B,D,V", [(1, 256, 3000), (37, 1536, 20001), (130, 192, 4097)])
def test_decode_step(B, D, V):
    X, w, W, u = make(1, B, D, V)
    head, kw = cce.Fp8Head.from_dense(W), settings(B)
    buf = cce.DecodeBuffers.alloc(B, head)
    cce.decode_step(X, w, EPS, head, u, buf, **kw)
    torch.cuda.synchronize()
    assert cce.cce_device_status(buf.ws) == 0
    # the logits: the product of the 8-bit operands, and near the exact head's
    a = O.rows_values(f64(buf.H8), buf.Hs.cpu().numpy())
    b = O.blocks_values(f64(head.q), head.s.cpu().numpy())
    want, size = a @ b.T, np.abs(a) @ np.abs(b).T
    l = f64(buf.logits)
    assert (np.abs(l - want) <= (2.0 ** -16 + (O.groups(D) + 4) * 2.0 ** -24) * size).all()
    exact = O.norm_forward(f64(X), f64(w), EPS)[0] @ f64(W).T
    # each factor is within 2^-4 of its value, elements apart: |error| below
    # (2^-3 + 2^-8) times the sum of magnitudes
    assert (np.abs(l - exact) <= (2.0 ** -3 + 2.0 ** -7) * size * 1.2).all()
    k = {n: v.cpu().numpy() for n, v in kw.items()}
    for r in range(B):
        tok, lp, _ = O.sample_row(l[r], float(k["temperature"][r]), int(k["top_k"][r]),
                                  float(k["top_p"][r]), float(k["min_p"][r]), float(u[r]))
        assert int(buf.tokens[r]) == tok
        assert abs(float(buf.logp[r]) - lp) <= 1e-5 * max(1.0, abs(lp))


@pytest.mark.parametrize("frozen", [False, True])
@pytest.mark.parametrize("split,D,V", [((16, 40, 33), 256, 3000), ((100, 520, 500), 256, 2100)])
def test_sampled_tokens_train_through_the_checkpoint(split, D, V, frozen):
    P, Rc, Rr = split
    M = sum(split)
    X, w, W, u = make(2, M, D, V)
    # label the response rows with sampled tokens
    h8 = cce.Fp8Head.from_dense(W)
    dec = cce.DecodeBuffers.alloc(M, h8)
    cce.decode_step(X, w, EPS, h8, u, dec)
    labels = dec.tokens.clone()
    labels[0] = -1
    head = cce.Head(w=W, V=V, D=D)
    layout = (0, P, P, P + Rc, P + Rc, M)
    norm = cce.NormBuffers.alloc(M, D, frozen=frozen)
    buf = cce.HeadBuffers.alloc(M, D, V, cce.CCE_BF16, head)
    cce.orpo_norm_head_pass(X, w, EPS, head, labels, layout, 0.1, "full", 0.0, False, norm, buf)
    torch.cuda.synchronize()
    assert cce.cce_device_status(buf.ws) == 0
    y = labels.cpu().numpy()
    H, rstd = f64(norm.H), f64(norm.rstd)
    L = F.Layout(*layout)
    logp, lse, _ = F.head_forward(H, f64(W), y)
    o = F.orpo_loss_from_logps(logp, y, L, 0.1, "full")
    g = F.orpo_grad_coeffs(logp, y, L, 0.1, "full")
    dH = F.head_dh(H, f64(W), y, g, lse)
    n = O.rows_values(f64(norm.X8), norm.Xs.cpu().numpy()) * rstd[:, None]
    dX, dW = O.norm_backward(n, rstd, f64(w), dH)
    assert np.abs(f64(buf.logp) - logp).max() <= TOL_LOGP
    assert abs(float(buf.out8[0]) - o.loss) <= TOL_LOSS * abs(o.loss)
    assert rel_fro(f64(norm.dX), dX) <= TOL_DH
    if not frozen:
        assert rel_fro(f64(norm.dW), dW) <= TOL_DH
    # against the gradient without a checkpoint: x enters through n alone,
    # whose elements are off by at most 2^-4
    full, full_w = O.norm_backward(f64(X) * rstd[:, None], rstd, f64(w), dH)
    assert rel_fro(f64(norm.dX), full) <= 2.0 ** -3 and (frozen or rel_fro(dW, full_w) <= 2.0 ** -3)
    # the 8-bit head that sampled and the dense head that trains agree on the
    # sampled tokens' log-probs to the operands' rounding
    assert np.median(np.abs(f64(dec.logp) - F.head_forward(H, f64(W), dec.tokens.cpu().numpy())[0])) < 0.25


def test_both_in_graphs():
    """Captured once, replayed on new inputs: the same bits as direct calls."""
    M, D, V = 64, 512, 5000
    X, w, W, u = make(3, M, D, V)
    head, h8 = cce.Head(w=W, V=V, D=D), cce.Fp8Head.from_dense(W)
    layout, kw = (0, 10, 10, 40, 40, M), settings(M)

    def bufs():
        return (cce.DecodeBuffers.alloc(M, h8), cce.NormBuffers.alloc(M, D),
                cce.HeadBuffers.alloc(M, D, V, cce.CCE_BF16, head))

    def run(dec, norm, buf):
        cce.decode_step(X, w, EPS, h8, u, dec, **kw)
        cce.orpo_norm_head_pass(X, w, EPS, head, dec.tokens, layout, 0.1, "response", 0.0, False,
                                norm, buf)

    a, b = bufs(), bufs()
    run(*a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run(*b)
    X2, _, _, u2 = make(4, M, D, V)
    X.copy_(X2)
    u.copy_(u2)
    graph.replay()
    torch.cuda.synchronize()
    run(*a)
    torch.cuda.synchronize()
    for x, y in ((a[0].tokens, b[0].tokens), (a[0].logp, b[0].logp), (a[0].logits, b[0].logits),
                 (a[1].dX, b[1].dX), (a[1].dW, b[1].dW), (a[2].out8, b[2].out8)):
        assert torch.equal(x, y)
    assert cce.cce_device_status(a[2].ws) == 0 and cce.cce_device_status(b[2].ws) == 0


FIRST_IN_A_CAPTURE = """
import torch
from lm_head_cross_flash_b200 import cce
B, D, V = {B}, 256, 30000
X, w = torch.randn(B, D, device="cuda"), torch.ones(D, device="cuda")
W, u = torch.randn(V, D, device="cuda"), torch.full((B,), 0.5, device="cuda")
q, s = cce.fp8_empty(V, D), torch.empty(cce.fp8_groups(V), cce.fp8_groups(D), device="cuda")
head = cce.Fp8Head(q, s)
buf, norm = cce.DecodeBuffers.alloc(B, head), cce.NormBuffers.alloc(B, D, cce.CCE_F32, torch.float32)
dH = torch.ones(B, D, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    cce.cce_fp8_quant_blocks(W, q, s)
    cce.decode_step(X, w, 1e-6, head, u, buf, top_p=torch.full((B,), 0.9, device="cuda"))
    cce.cce_norm_forward(X, w, 1e-6, norm.H, X8=norm.X8, Xs=norm.Xs, rstd=norm.rstd)
    cce.cce_norm_backward(norm.X8, norm.Xs, norm.rstd, w, dH, norm.dX, norm.dW, norm.ws)
g.replay()
torch.cuda.synchronize()
tokens, dX = buf.tokens.clone(), norm.dX.clone()
cce.decode_step(X, w, 1e-6, head, u, buf, top_p=torch.full((B,), 0.9, device="cuda"))
cce.cce_norm_backward(norm.X8, norm.Xs, norm.rstd, w, dH, norm.dX, norm.dW, norm.ws)
torch.cuda.synchronize()
assert torch.equal(tokens, buf.tokens) and torch.equal(dX, norm.dX) and (tokens >= 0).all()
print("captured")
"""


@pytest.mark.parametrize("B", [3, 200])
def test_the_first_calls_of_a_process_may_be_captured(B):
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_IN_A_CAPTURE.replace("{B}", str(B))],
                       capture_output=True, text=True, cwd=root, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_two_streams_at_once():
    """Two decoding steps on two streams, each with buffers of its own."""
    D, V = 512, 30000
    X, w, W, u = make(5, 8, D, V)
    h8 = cce.Fp8Head.from_dense(W)
    bufs = [cce.DecodeBuffers.alloc(8, h8) for _ in range(3)]
    cce.decode_step(X, w, EPS, h8, u, bufs[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for s, b in zip(streams, bufs[1:]):
            cce.decode_step(X, w, EPS, h8, u, b, stream=s)
    torch.cuda.synchronize()
    for b in bufs[1:]:
        assert torch.equal(b.tokens, bufs[0].tokens) and torch.equal(b.logp, bufs[0].logp)
        assert torch.equal(b.logits, bufs[0].logits)


def far(x):
    """The same values with rows 2^30 elements apart: offsets pass 32 bits."""
    rows, cols = x.shape
    y = torch.empty((rows - 1) * 2 ** 30 + cols, dtype=x.dtype, device="cuda")
    y = y.as_strided((rows, cols), (2 ** 30, 1))
    y.copy_(x)
    return y


def test_rows_far_apart():
    """Every matrix with a row stride of 2^30 gives what dense rows give."""
    M, D, V = 4, 256, 3000
    X, w, W, u = make(6, M, D, V)
    G = cce.fp8_groups(D)
    f32 = lambda *s: torch.empty(*s, device="cuda")
    codes = lambda r, c: cce.fp8_empty(r, c).zero_()

    def run(wrap):
        x, h = wrap(X), wrap(torch.zeros_like(X))
        x8, xs, rstd, h8, hs = wrap(codes(M, D)), f32(M, G), f32(M), wrap(codes(M, D)), f32(M, G)
        cce.cce_norm_forward(x, w, EPS, h, h8, hs, x8, xs, rstd)
        dh, dx, dw = wrap(X.float()), wrap(torch.zeros_like(X)), f32(D)
        ws = torch.zeros(cce.cce_norm_backward_workspace_bytes(M, D), dtype=torch.uint8, device="cuda")
        cce.cce_norm_backward(x8, xs, rstd, w, dh, dx, dw, ws)
        q, s = wrap(codes(M, D)), f32(M, G)
        cce.cce_fp8_quant_rows(x, q, s)
        wq, wsc = wrap(codes(M, D)), f32(1, G)
        cce.cce_fp8_quant_blocks(x, wq, wsc)
        few, st = wrap(torch.zeros(M, M, device="cuda")), torch.zeros(256, dtype=torch.uint8, device="cuda")
        cce.cce_fp8_matmul(h8, hs, wq, wsc, few, st)
        head = cce.Fp8Head.from_dense(W)
        logits = wrap(torch.zeros(M, V, device="cuda"))
        cce.cce_fp8_matmul(h8, hs, head.q, head.s, logits, st)
        tok, lp = torch.zeros(M, dtype=torch.int32, device="cuda"), f32(M)
        cce.cce_sample_rows(logits, None, None, torch.full((M,), 0.9, device="cuda"), None, u[:M], tok, lp)
        torch.cuda.synchronize()
        return [t.float().cpu() for t in (h, x8, xs, rstd, h8, hs, dx, dw, q, s, wq, wsc, few, logits, tok, lp)]

    for a, b in zip(run(lambda t: t), run(far)):
        assert torch.equal(a, b)
    # the many-rows product: C's rows far apart (130 rows would need 520 GB at
    # that stride, so theirs is 2^25: the last row begins beyond 2^32)
    A, B = make(7, 130, D, 200)[0], make(8, 10, D, 200)[2]
    a8, sa = codes(130, D), f32(130, G)
    cce.cce_fp8_quant_rows(A, a8, sa)
    hb = cce.Fp8Head.from_dense(B)
    st = torch.zeros(256, dtype=torch.uint8, device="cuda")
    dense, wide = f32(130, 200), torch.empty(129 * 2 ** 25 + 200, device="cuda").as_strided((130, 200), (2 ** 25, 1))
    cce.cce_fp8_matmul(a8, sa, hb.q, hb.s, dense, st)
    cce.cce_fp8_matmul(a8, sa, hb.q, hb.s, wide, st)
    assert torch.equal(dense, wide)


def test_a_head_made_on_another_stream():
    """The codes' memory may still be written by the current stream's earlier
    work (a tensor freed behind it), and so may the dense head: a head made on
    another stream comes behind both."""
    V, D = 4096, 512
    _, _, W, _ = make(9, 1, D, V)
    want = cce.Fp8Head.from_dense(W)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    late = torch.zeros_like(W)
    torch.cuda.synchronize()
    for _ in range(3):
        q, s = torch.empty(V, D, dtype=torch.uint8, device="cuda"), torch.empty(V // 128, D // 128, device="cuda")
        torch.cuda._sleep(20_000_000)  # some 10 ms
        q.fill_(0x11)
        s.fill_(3.0)
        late.copy_(W)
        del q, s
        got = cce.Fp8Head.from_dense(late, stream=side)
        side.synchronize()
        assert torch.equal(got.q.view(torch.uint8), want.q.view(torch.uint8)) and torch.equal(got.s, want.s)
        torch.cuda.synchronize()
        late.zero_()
        del got
