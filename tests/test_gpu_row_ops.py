"""8-bit quantisation and the final norm (forward, checkpoint, backward) on
the GPU against the float64 oracle.

Tolerances, derived from the arithmetic (u = 2^-24, fp32 half step):
* codes and scales: exact (the format fixes every rounding);
* H: the sum of squares is a chain of at most 32 fused adds, 10 tree adds, so
  at most 42 u relative, half of that in rstd; eps, quotient, root and the two
  products add less than 8 u.  32 u in all, plus the output's own half step
  (2^-8 for bf16);
* dX: g has one rounding, n two, the dot product at most 32 + 10 chained adds
  of terms with three roundings, and the result four more operations:
  rstd (6 u |g| + 56 u |n| mean|g n|), plus the output's half step;
* dW: a sum of M terms in some order, each with three roundings:
  (M + 4) u sum|dH n|.
"""

import numpy as np
import pytest
import torch

from lm_head_cross_flash_b200 import cce
from oracle import head_ops as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
T = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": U, "bf16": 2.0 ** -8}


def rows(seed, M, D, dtype, pad=0, scale=1.0):
    """A [M, D] view with `pad` more columns behind each row."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((M, D + pad)) * np.exp(0.5 * r.standard_normal((M, 1))) * scale
    x[:, r.integers(0, D, max(1, D // 256))] *= 20.0
    return torch.from_numpy(x.astype(np.float32)).cuda().to(T[dtype])[:, :D]


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def codes(rows_, cols, pad=0):
    q = torch.full((rows_, cols + pad), 1.0, device="cuda").to(torch.float8_e4m3fn)
    return q[:, :cols]


def f32(*shape):
    return torch.full(shape, float("nan"), dtype=torch.float32, device="cuda")


SHAPES = [(1, 1, 0), (1, 128, 0), (3, 127, 1), (5, 129, 7), (17, 200, 56), (2, 2048, 0),
          (33, 1536, 8), (3, 4096, 0), (2, 8200, 3), (1, 16384, 0)]
# more rows than run at once: blocks take several
MANY = [(4001, 200, 0), (3001, 512, 0), (1501, 1000, 24), (700, 4096, 0), (350, 8200, 0), (700, 2047, 1)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,D,pad", SHAPES + [(5001, 1100, 4), (40003, 72, 0)])
def test_quant_rows_is_exact(M, D, pad, dtype):
    x = rows(1, M, D, dtype, pad)
    q, s = codes(M, D, pad), f32(M, O.groups(D))
    cce.cce_fp8_quant_rows(x, q, s)
    qo, so = O.quant_rows(x.float().cpu().numpy())
    assert np.array_equal(f64(q), qo)
    assert np.array_equal(s.cpu().numpy(), so)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,K,pad", [(1, 1, 0), (128, 128, 0), (129, 127, 1), (300, 1000, 24),
                                     (127, 513, 3), (1000, 256, 0)])
def test_quant_blocks_is_exact(N, K, pad, dtype):
    x = rows(2, N, K, dtype, pad, 0.02)
    q, s = codes(N, K, pad), f32(O.groups(N), O.groups(K))
    cce.cce_fp8_quant_blocks(x, q, s)
    qo, so = O.quant_blocks(x.float().cpu().numpy())
    assert np.array_equal(f64(q), qo)
    assert np.array_equal(s.cpu().numpy(), so)


def test_quant_edge_values():
    """Zero groups, the smallest and largest magnitudes, ties, NaN and
    infinities."""
    x = np.zeros((8, 256), np.float32)
    x[1, :128] = np.float32(1e-40)
    x[2] = np.linspace(-1, 1, 256) * 3.0e38
    x[3, 0] = 448.0
    x[3, 1:17] = np.arange(16) * 0.5 + 16.0   # halfway points of the codes
    x[4, 5], x[4, 6] = np.nan, 2.0
    x[5, 7], x[5, 200] = np.inf, 3.0
    x[6, :128] = np.nan
    x[7] = np.float32(2.0 ** -126)
    t = torch.from_numpy(x).cuda()
    q, s = codes(8, 256), f32(8, 2)
    cce.cce_fp8_quant_rows(t, q, s)
    qo, so = O.quant_rows(x)
    assert np.array_equal(s.cpu().numpy(), so)
    assert np.array_equal(f64(q), qo, equal_nan=True)
    with np.errstate(invalid="ignore"):
        v = f64(q) * np.repeat(s.cpu().numpy().astype(np.float64), 128, 1)
    assert np.isnan(v[4, 5]) and np.isfinite(np.delete(v[4], 5)).all()
    assert np.isnan(v[5, :128]).all() and np.isfinite(v[5, 128:]).all()
    assert (v[0] == 0).all()


@pytest.mark.parametrize("xt,wt,ht", [("bf16", "bf16", "bf16"), ("f32", "f32", "f32"),
                                      ("bf16", "f32", "bf16"), ("f32", "bf16", "bf16")])
@pytest.mark.parametrize("M,D,pad", SHAPES + MANY)
def test_norm_forward(M, D, pad, xt, wt, ht):
    x, w = rows(3, M, D, xt, pad), rows(4, 1, D, wt)[0].contiguous()
    G = O.groups(D)
    h = torch.full((M, D + pad), 7.0, dtype=T[ht], device="cuda")
    h8, hs, x8, xs = codes(M, D, pad), f32(M, G), codes(M, D, pad), f32(M, G)
    rstd = f32(M)
    cce.cce_norm_forward(x, w, 1e-6, h[:, :D], h8, hs, x8, xs, rstd)
    ho, ro = O.norm_forward(f64(x), f64(w), 1e-6)
    assert (np.abs(f64(rstd) - ro) <= 32 * U * ro).all()
    assert (np.abs(f64(h)[:, :D] - ho) <= (32 * U + HALF[ht]) * np.abs(ho)).all()
    if pad:
        assert (h[:, D:] == 7.0).all()
    qo, so = O.quant_rows(x.float().cpu().numpy())
    assert np.array_equal(f64(x8), qo) and np.array_equal(xs.cpu().numpy(), so)
    # the 8-bit rows of H: each value within a code's half step of H
    big = np.repeat(f64(hs), 128, 1)[:, :D]
    v = f64(h8) * big
    assert (np.abs(v - ho) <= np.maximum(2.0 ** -4 * np.abs(ho), 2.0 ** -10 * big) * (1 + 2.0 ** -16)
            ).all()
    # every subset of the outputs gives the same values
    h2, r2, q2, s2 = torch.empty_like(h), f32(M), codes(M, D, pad), f32(M, G)
    cce.cce_norm_forward(x, w, 1e-6, H=h2[:, :D])
    cce.cce_norm_forward(x, w, 1e-6, rstd=r2)
    cce.cce_norm_forward(x, w, 1e-6, H8=q2, Hs=s2)
    assert torch.equal(h2[:, :D], h[:, :D]) and torch.equal(r2, rstd)
    assert torch.equal(q2.view(torch.uint8), h8.view(torch.uint8)) and torch.equal(s2, hs)


@pytest.mark.parametrize("dht,dxt,wt", [("f32", "bf16", "bf16"), ("f32", "f32", "f32"),
                                        ("bf16", "bf16", "f32"), ("bf16", "f32", "bf16")])
@pytest.mark.parametrize("M,D,pad", SHAPES + MANY + [(601, 256, 0), (700, 40, 0), (400, 2048, 0)])
def test_norm_backward(M, D, pad, dht, dxt, wt):
    x, w = rows(5, M, D, "f32"), rows(6, 1, D, wt)[0].contiguous()
    dh = rows(7, M, D, dht, pad, 1e-3)
    x8, xs, rstd = codes(M, D, pad), f32(M, O.groups(D)), f32(M)
    cce.cce_norm_forward(x, w, 1e-6, X8=x8, Xs=xs, rstd=rstd)
    dx = torch.full((M, D + pad), 7.0, dtype=T[dxt], device="cuda")
    dw = f32(D)
    n_ws = cce.cce_norm_backward_workspace_bytes(M, D)
    ws = torch.full((n_ws + 64,), 0x5A, dtype=torch.uint8, device="cuda")
    cce.cce_norm_backward(x8, xs, rstd, w, dh, dx[:, :D], dw, ws[:n_ws])
    assert (ws[n_ws:] == 0x5A).all()
    r = f64(rstd)
    n = O.rows_values(f64(x8), xs.cpu().numpy()) * r[:, None]
    d64, w64 = f64(dh), f64(w)
    dxo, dwo = O.norm_backward(n, r, w64, d64)
    g = d64 * w64
    tol = r[:, None] * U * (6 * np.abs(g) + 56 * np.abs(n) * np.abs(g * n).mean(1, keepdims=True))
    assert (np.abs(f64(dx)[:, :D] - dxo) <= tol + HALF[dxt] * (np.abs(dxo) + tol)).all()
    assert (np.abs(f64(dw) - dwo) <= (M + 4) * U * np.abs(d64 * n).sum(0)).all()
    if pad:
        assert (dx[:, D:] == 7.0).all()
    # frozen norm: no dW, no workspace, the same dX; and the same bits again
    dx2, dw2 = torch.full_like(dx, 7.0), f32(D)
    cce.cce_norm_backward(x8, xs, rstd, w, dh, dx2[:, :D])
    assert torch.equal(dx2, dx)
    cce.cce_norm_backward(x8, xs, rstd, w, dh, dx2[:, :D], dw2, ws[:n_ws])
    assert torch.equal(dx2, dx) and torch.equal(dw2, dw)


def test_norm_backward_against_differences():
    """dX is the slope of sum(dH * H) in x, taken by central differences of
    the oracle's forward around the checkpointed rows."""
    M, D = 3, 160
    x = rows(8, M, D, "f32")
    w = rows(9, 1, D, "f32")[0].contiguous()
    x8, xs, rstd = codes(M, D), f32(M, 2), f32(M)
    cce.cce_fp8_quant_rows(x, x8, xs)
    xr = O.rows_values(f64(x8), xs.cpu().numpy())
    _, r = O.norm_forward(xr, f64(w), 1e-6)
    rstd.copy_(torch.from_numpy(r))
    dh = rows(10, M, D, "f32")
    dx, dw = torch.empty(M, D, device="cuda"), f32(D)
    ws = torch.zeros(cce.cce_norm_backward_workspace_bytes(M, D), dtype=torch.uint8, device="cuda")
    cce.cce_norm_backward(x8, xs, rstd, w, dh, dx, dw, ws)
    rng = np.random.default_rng(11)
    for _ in range(20):
        v, vw = rng.standard_normal((M, D)), rng.standard_normal(D)
        h = 1e-5

        def f(a, b):
            return float((f64(dh) * O.norm_forward(xr + a * v, f64(w) + b * vw, 1e-6)[0]).sum())

        num, numw = (f(h, 0) - f(-h, 0)) / (2 * h), (f(0, h) - f(0, -h)) / (2 * h)
        # central differences: h^2 times the third derivative, below 1e-7 of the
        # terms' sizes here; the kernel's own error is below 64 u of them
        size = np.abs(f64(dx) * v).sum() + np.abs(f64(dh) * f64(w) * xr).sum() * r.max()
        assert abs(num - float((f64(dx) * v).sum())) <= 1e-5 * size
        assert abs(numw - float((f64(dw) * vw).sum())) <= 1e-5 * np.abs(f64(dw) * vw).sum() + 1e-6


def test_norm_rows_of_zero_and_dead_gradient_rows():
    x = torch.zeros(4, 256, device="cuda")
    x[1] = 1.0
    w = torch.ones(256, device="cuda")
    x8, xs, rstd, h = codes(4, 256), f32(4, 2), f32(4), f32(4, 256)
    cce.cce_norm_forward(x, w, 1e-6, h, X8=x8, Xs=xs, rstd=rstd)
    assert torch.isfinite(h).all() and (h[0] == 0).all()
    dh = torch.zeros(4, 256, device="cuda")
    dh[1] = 1.0
    dx, dw = f32(4, 256), f32(256)
    ws = torch.zeros(cce.cce_norm_backward_workspace_bytes(4, 256), dtype=torch.uint8, device="cuda")
    cce.cce_norm_backward(x8, xs, rstd, w, dh, dx, dw, ws)
    assert (dx[0] == 0).all() and (dx[2:] == 0).all() and torch.isfinite(dw).all()


def test_another_stream_and_a_graph():
    M, D = 65, 1536
    x, w = rows(12, M, D, "bf16"), rows(13, 1, D, "bf16")[0].contiguous()
    G = O.groups(D)
    dh = rows(14, M, D, "f32", 0, 1e-3)

    def bufs():
        return dict(h=torch.zeros(M, D, dtype=torch.bfloat16, device="cuda"), x8=codes(M, D),
                    xs=f32(M, G), rstd=f32(M), dx=torch.zeros(M, D, dtype=torch.bfloat16, device="cuda"),
                    dw=f32(D), ws=torch.zeros(cce.cce_norm_backward_workspace_bytes(M, D),
                                              dtype=torch.uint8, device="cuda"))

    def step(b, stream=None):
        cce.cce_norm_forward(x, w, 1e-6, b["h"], X8=b["x8"], Xs=b["xs"], rstd=b["rstd"],
                             stream=stream)
        cce.cce_norm_backward(b["x8"], b["xs"], b["rstd"], w, dh, b["dx"], b["dw"], b["ws"],
                              stream=stream)

    a, b, c = bufs(), bufs(), bufs()
    step(a)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    step(b, side)
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(c)
    x.copy_(rows(15, M, D, "bf16"))  # replayed on new inputs
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)) for k in ("h", "x8", "dx", "dw"))
    assert not torch.equal(c["h"], a["h"])
    step(a)
    torch.cuda.synchronize()
    assert all(torch.equal(a[k].view(torch.uint8), c[k].view(torch.uint8)) for k in ("h", "x8", "dx", "dw"))
