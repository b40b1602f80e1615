"""The 8-bit blocked product on the GPU against the float64 oracle.

Tolerance.  Inside a group the 128 products of two e4m3 values (8-bit
significands) are exact in fp32 and are summed by the tensor cores in fp32; a
sum of 128 terms is off by at most 128 truncations of 2^-23 of the largest
partial sum, 2^-16 sum|a b|.  The scales' product and the FMA add (3 + G) 2^-24
of sum_g |sa sb| sum|a b| over the G groups.  In all (2^-16 + (G + 3) 2^-24)
times that sum, and the output's half step (2^-8 for bf16).
"""

import numpy as np
import pytest
import torch

from lm_head_cross_flash_b200 import cce
from oracle import head_ops as O

pytestmark = pytest.mark.gpu

T = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def operand(seed, rows, K, kind, dist="normal", pad=0):
    """Codes with rows on 16-byte boundaries and NaN codes in the padding."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((rows, K)) if dist == "normal" else r.uniform(0.5, 1.5, (rows, K))
    x = torch.from_numpy((x * np.exp(r.standard_normal((rows, 1)))).astype(np.float32)).cuda()
    ld = -(-K // 16) * 16 + pad
    q = torch.full((rows, ld), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)[:, :K]
    G = O.groups(K)
    s = torch.empty(rows if kind == "rows" else O.groups(rows), G, device="cuda")
    (cce.cce_fp8_quant_rows if kind == "rows" else cce.cce_fp8_quant_blocks)(x, q, s)
    v = O.rows_values if kind == "rows" else O.blocks_values
    return q, s, v(q.float().cpu().numpy(), s.cpu().numpy())


def check(c, av, bv, K, half):
    want, size = av @ bv.T, np.abs(av) @ np.abs(bv).T
    tol = (2.0 ** -16 + (O.groups(K) + 3) * 2.0 ** -24) * size
    err = np.abs(c.float().cpu().numpy().astype(np.float64) - want)
    bad = err > tol + half * (np.abs(want) + tol)
    assert not bad.any(), (np.argwhere(bad)[:5].tolist(), float((err / size).max()))


@pytest.fixture
def ws():
    return torch.zeros(256, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("ct", ["bf16", "f32"])
@pytest.mark.parametrize("M", [1, 2, 16, 17, 33, 64, 65, 128, 129, 300])
@pytest.mark.parametrize("N,K", [(1, 1), (127, 128), (129, 100), (1000, 1029), (4096, 512), (520, 2048)])
def test_product(M, N, K, ct, ws):
    a, sa, av = operand(1, M, K, "rows")
    b, sb, bv = operand(2, N, K, "blocks")
    big = torch.full((M, N + 5), 7.0, dtype=T[ct], device="cuda")
    cce.cce_fp8_matmul(a, sa, b, sb, big[:, :N], ws)
    assert cce.cce_device_status(ws) == 0
    check(big[:, :N], av, bv, K, HALF[ct])
    assert (big[:, N:] == 7.0).all()


@pytest.mark.parametrize("M", [3, 100, 260])
def test_product_of_one_sign(M, ws):
    """Sums that grow over all of K, with row strides of their own and an
    output whose rows start on 16-byte boundaries."""
    N, K = 384, 4000
    a, sa, av = operand(3, M, K, "rows", "positive", 64)
    b, sb, bv = operand(4, N, K, "blocks", "positive", 32)
    for ct in ("f32", "bf16"):
        c = torch.empty(M, N + 64, dtype=T[ct], device="cuda")[:, :N]
        cce.cce_fp8_matmul(a, sa, b, sb, c, ws)
        check(c, av, bv, K, HALF[ct])


def test_long_inner_dimension(ws):
    """K = 65,536: the few-rows kernel has no room for its scales."""
    for M, N in ((1, 130), (100, 200), (100, 20000)):
        a, sa, av = operand(5, M, 65536, "rows")
        b, sb, bv = operand(6, N, 65536, "blocks") if N < 1000 else operand(6, 300, 65536, "blocks")
        c = torch.empty(M, b.shape[0], device="cuda")
        cce.cce_fp8_matmul(a, sa, b, sb, c, ws)
        check(c, av, bv, 65536, HALF["f32"])


def test_many_tiles_per_cta(ws):
    """More tiles than SMs, on both kernels; rows of zeros stay zero."""
    K = 256
    b, sb, bv = operand(7, 40000, K, "blocks")
    for M in (5, 64, 700):
        a, sa, av = operand(8, M, K, "rows")
        sa[0] = 0.0
        av[0] = 0.0
        c = torch.full((M, 40000), 7.0, dtype=torch.bfloat16, device="cuda")
        cce.cce_fp8_matmul(a, sa, b, sb, c, ws)
        check(c, av, bv, K, HALF["bf16"])
        assert (c[0] == 0).all()
    assert cce.cce_device_status(ws) == 0


def test_rounds_once_and_repeats_its_bits(ws):
    a, sa, _ = operand(9, 40, 1536, "rows")
    b, sb, _ = operand(10, 5000, 1536, "blocks")
    c32, c16, again = (torch.empty(40, 5000, device="cuda"),
                       torch.empty(40, 5000, dtype=torch.bfloat16, device="cuda"),
                       torch.empty(40, 5000, device="cuda"))
    cce.cce_fp8_matmul(a, sa, b, sb, c32, ws)
    cce.cce_fp8_matmul(a, sa, b, sb, c16, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cce.cce_fp8_matmul(a, sa, b, sb, again, ws, side)
    side.synchronize()
    assert torch.equal(c32.bfloat16(), c16) and torch.equal(c32, again)
    g = torch.cuda.CUDAGraph()
    out = torch.zeros_like(c32)
    with torch.cuda.graph(g):
        cce.cce_fp8_matmul(a, sa, b, sb, out, ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, c32)


@pytest.mark.parametrize("M,N,K", [(100, 9500, 8192), (100, 9500, 8193), (128, 9500, 8320),
                                   (65, 20000, 8321), (33, 9500, 16385), (100, 2600, 33000)])
def test_few_rows_whose_scales_do_not_fit(M, N, K, ws):
    """The few-rows kernel keeps a CTA's scales in shared memory, 8,192 of
    them: M padded to 16, 32, 64 or 128, times the groups of K that a CTA takes
    (all of them where the head has 75 tiles of 128 rows or more, else a share
    of 1/2, 1/4 or 1/8).  Just below that (the first case) it runs; with one
    group more, up to 128 rows go to the many-rows kernel, whose tiles are
    taller than the operand."""
    G, tiles = O.groups(K), O.groups(N)
    split = 1
    while split < 8 and 2 * split * tiles <= 148 and 2 * split <= G:
        split *= 2
    scales = (64 if M <= 64 else 128) * -(-G // split)
    assert (scales <= 8192) == ((M, K) == (100, 8192))
    a, sa, av = operand(11, M, K, "rows")
    b, sb, bv = operand(12, N, K, "blocks")
    for ct in ("f32", "bf16"):
        big = torch.full((M + 1, N + 3), 7.0, dtype=T[ct], device="cuda")
        cce.cce_fp8_matmul(a, sa, b, sb, big[:M, :N], ws)
        assert cce.cce_device_status(ws) == 0
        check(big[:M, :N], av, bv, K, HALF[ct])
        assert (big[:M, N:] == 7.0).all() and (big[M:] == 7.0).all()
