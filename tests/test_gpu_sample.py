"""Row sampling on the GPU against the float64 oracle.

Tokens are compared for equality: the running masses of the two differ by a
few 2^-45 of the largest weight a token, so a number u chosen without regard
to the row decides otherwise with a probability below 1e-8 a row.  logp: the
sum of the other weights is made of fp32 exponentials, each off by 2^-22 and
by its argument's rounding (at most 104 * 2^-24 where it does not vanish), so
|error| <= 7e-6 min(1, sum) plus the output's half step, 2^-24 relative.
"""

import numpy as np
import pytest
import torch

from lm_head_cross_flash_b200 import cce
from oracle import head_ops as O

pytestmark = pytest.mark.gpu


def t32(x, dtype=torch.float32):
    return torch.tensor(np.asarray(x), dtype=dtype, device="cuda")


def run(l, t=None, k=None, p=None, mp=None, u=None, with_logp=True, stream=None):
    B = l.shape[0]
    tok = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    lp = torch.full((B,), float("nan"), device="cuda") if with_logp else None
    cce.cce_sample_rows(l, None if t is None else t32(t), None if k is None else t32(k, torch.int32),
                        None if p is None else t32(p), None if mp is None else t32(mp),
                        t32(u), tok, lp, stream)
    torch.cuda.synchronize()
    return tok.cpu().numpy(), None if lp is None else lp.cpu().numpy()


def check(l, t=None, k=None, p=None, mp=None, u=None):
    B = l.shape[0]
    tok, lp = run(l, t, k, p, mp, u)
    x = l.float().cpu().numpy().astype(np.float64)
    f = lambda v, d: np.full(B, d) if v is None else np.asarray(v)
    t, k, p, mp = f(t, 1.0), f(k, 0), f(p, 1.0), f(mp, 0.0)
    u = np.asarray(u)
    for r in range(B):
        g = lambda v: float(np.float32(v[r]))
        want, wlp, _ = O.sample_row(x[r], g(t), int(k[r]), g(p), g(mp), g(u))
        what = (r, g(t), int(k[r]), g(p), g(mp), g(u))
        assert tok[r] == want, (what, tok[r], want)
        rest = 0.0 if want < 0 else np.expm1(-min(wlp, 0.0)) if tok[r] == np.nanargmax(x[r]) else 1.0
        assert abs(lp[r] - wlp) <= 7e-6 * min(1.0, rest) + 2.0 ** -24 * abs(wlp) + 1e-30, (what, lp[r], wlp)
    return tok


def logits(seed, B, V, dtype, spread=2.5, peaks=True, masked=0.0, pad=0):
    r = np.random.default_rng(seed)
    x = spread * r.standard_normal((B, V + pad))
    if peaks:
        for b in range(B):
            n = min(V, 40)
            x[b, r.integers(0, V, n)] = spread * (4 + 1.5 * r.uniform(0.2, 1.2) * r.exponential(size=n))
    if masked:
        x[r.random(x.shape) < masked] = -np.inf
    return t32(x).to(dtype)[:, :V]


def settings(seed, B):
    r = np.random.default_rng(seed)
    return dict(t=r.choice([0.0, 0.3, 0.7, 1.0, 1.0, 1.5, 3.0], B),
                k=r.choice([0, 0, 1, 2, 20, 50, 500, 3000, 10 ** 6], B),
                p=r.choice([1.0, 1.0, 0.0, 0.1, 0.5, 0.9, 0.95, 0.999], B),
                mp=r.choice([0.0, 0.0, 0.01, 0.1, 0.5, 1.0], B), u=r.random(B).astype(np.float32))


BF, F = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 63, 1000, 4097, 8192])
@pytest.mark.parametrize("masked", [0.0, 0.5, 0.99])
def test_small_vocabularies(V, dtype, masked):
    B = 40
    check(logits(V, B, V, dtype, masked=masked), **settings(V + 1, B))


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("B,V,spread,peaks", [(1, 73440, 2.5, True), (3, 128256, 1.0, False),
                                              (24, 50001, 4.0, True), (10, 262144, 1.0, False),
                                              (40, 32000, 0.1, False), (160, 20000, 2.5, True)])
def test_large_vocabularies(B, V, spread, peaks, dtype):
    l = logits(V, B, V, dtype, spread, peaks, pad=3)
    for seed in range(3 if B < 100 else 1):
        check(l, **settings(seed, B))
    n = np.random.default_rng(9).random(B).astype(np.float32)
    check(l, u=n)                       # plain
    check(l, p=[0.95] * B, u=n)         # nucleus alone
    check(l, mp=[0.02] * B, t=[1.3] * B, u=n)
    check(l, k=[50] * B, u=n)
    check(l, k=[V // 2] * B, p=[0.9] * B, u=n)


@pytest.mark.parametrize("B,V,spread,dtype", [(1500, 300, 2.5, BF), (400, 5000, 4.0, F),
                                              (350, 20000, 1.0, F), (200, 40001, 1.0, BF)])
def test_more_rows_than_run_at_once(B, V, spread, dtype):
    """Flat rows among others: the search's clusters take several rows each."""
    l = logits(V, B, V, dtype, spread, False)
    check(l, **settings(V, B))
    check(l, p=[0.9] * B, u=np.random.default_rng(2).random(B).astype(np.float32))


def test_rows_without_and_with_one_live_logit():
    l = torch.full((6, 5000), float("-inf"), device="cuda")
    l[1, 4999] = -1e30
    l[2, 17] = float("nan")
    l[3] = float("nan")
    l[4, 3], l[4, 4] = 5.0, float("nan")
    l[5, 0] = torch.finfo(F).min
    tok = check(l, t=[1.0] * 6, k=[0, 5, 0, 3, 0, 0], p=[0.9] * 6, mp=[0.1] * 6, u=[0.5] * 6)
    assert tok.tolist() == [-1, 4999, -1, -1, 3, 0]


def test_masks_of_the_lowest_value_stay_live():
    """A mask of the type's lowest finite value is a logit like others: it is
    chosen only where nothing else is."""
    for dtype in (F, BF):
        l = torch.full((3, 3000), torch.finfo(dtype).min, dtype=dtype, device="cuda")
        l[1, 100] = 0.0
        l[2, 5:8] = 1.0
        check(l, u=[0.5, 0.999, 0.9])
        check(l, k=[1000] * 3, p=[0.9] * 3, t=[2.0] * 3, u=[0.5, 0.999, 0.9])


def test_infinities_share_the_row():
    l = logits(5, 5, 2000, F)
    l[0, 7] = float("inf")
    l[1, [3, 900, 1999]] = float("inf")
    l[2] = float("inf")
    l[3, 1] = float("-inf")
    l[4, [2, 1000]] = float("inf")
    check(l, u=[0.4, 0.7, 0.123, 0.5, 0.9])
    check(l, k=[100] * 5, p=[0.6] * 5, mp=[0.5] * 5, t=[0.5] * 5, u=[0.4, 0.7, 0.123, 0.5, 0.9])


@pytest.mark.parametrize("V", [5, 2048, 2049, 40000, 300001])
def test_equal_logits(V):
    """One value, two values, and signed zeros: ranks go by index."""
    l = torch.zeros(4, V, device="cuda")
    l[1, ::2] = -0.0
    l[2, ::3] = 1.0
    l[3] = -3.25
    for u in (0.0, 0.25, 0.77, 0.9999):
        check(l, u=[u] * 4)
        check(l, k=[V // 2 + 1] * 4, u=[u] * 4)
        check(l, p=[0.5] * 4, u=[u] * 4)
        check(l, mp=[1.0] * 4, k=[0, 3, 0, V // 3 + 1], u=[u] * 4)


def test_few_values_many_ties():
    r = np.random.default_rng(3)
    l = t32(r.integers(0, 6, (6, 60000)) * 0.5)
    for s in range(3):
        check(l, **settings(s + 20, 6))


def test_extreme_ranges_and_temperatures():
    r = np.random.default_rng(4)
    x = r.standard_normal((8, 30000)) * np.array([1e-30, 1e-6, 1, 1e3, 1e10, 1e30, 3e37, 1e-3])[:, None]
    l = t32(x)
    for t in (1e-30, 1e-6, 0.05, 1.0, 50.0, 1e10, 3e38, float("inf")):
        check(l, t=[t] * 8, u=r.random(8).astype(np.float32))
        check(l, t=[t] * 8, k=[4000] * 8, p=[0.7] * 8, u=r.random(8).astype(np.float32))
        check(l, t=[t] * 8, mp=[0.3] * 8, u=r.random(8).astype(np.float32))


def test_long_tails_beyond_the_weights_range():
    """Mass far below the smallest weight, and targets next to the total."""
    V = 100000
    l = torch.linspace(0, -500, V, device="cuda").repeat(5, 1)
    l[1, 1:] -= 60.0
    l[2, 1:] -= 25.0
    l[3, V // 2:] = -1e30
    l[4] = l[4].flip(0)
    for u in (0.0, 0.5, 1.0 - 2.0 ** -24):
        for p in (1.0, 0.9999, 1.0 - 2.0 ** -24):
            check(l, p=[p] * 5, u=[u] * 5)
            check(l, p=[p] * 5, k=[60000] * 5, u=[u] * 5)


def test_numbers_outside_their_ranges():
    l = logits(6, 8, 3000, F)
    nan = float("nan")
    tok, _ = run(l, u=[-1.0, nan, 0.0, 1.0, 2.0, 1.0 - 2.0 ** -24, 0.5, 0.5],
                 t=[1, 1, 1, 1, 1, 1, nan, -2.0])
    a, _ = run(l, u=[0.0] * 3 + [1.0 - 2.0 ** -24] * 3 + [0.5] * 2, t=[1.0] * 6 + [0.0] * 2)
    assert (tok == a).all()
    check(l, u=[0.3] * 8, p=[-1.0, 0.0, 5.0, 1.0, 0.5, 0.5, 0.5, 0.5], k=[-3, 0, 2 ** 31 - 1] + [4] * 5,
          mp=[-1.0, 0.0, 2.0, 1.0] + [0.1] * 4)
    b, _ = run(l, u=[0.3] * 8, p=[nan] * 8, mp=[nan] * 8)
    c, _ = run(l, u=[0.3] * 8)
    assert (b == c).all()


def test_a_vocabulary_beyond_shared_memory():
    """V = 1,000,003: the slices are read from memory in every pass."""
    l = logits(7, 2, 1000003, F, 1.0, False)
    check(l, u=[0.2, 0.9])
    check(l, k=[40, 700000], p=[0.9, 0.99], u=[0.2, 0.9])


def test_the_draw_follows_the_probabilities():
    """Each token's share of evenly spaced numbers is its probability to
    within one spacing."""
    V, n = 50, 1000
    l = logits(8, 1, V, F, 1.0, False)
    tok, _ = run(l.expand(n, V).contiguous(), u=(np.arange(n) + 0.5) / n, with_logp=False)
    p = torch.softmax(l[0].double(), 0).cpu().numpy()
    assert (np.abs(np.bincount(tok, minlength=V) / n - p) <= 1.0 / n + 1e-12).all()


def test_repeats_on_a_stream_and_in_a_graph():
    l, s = logits(9, 33, 60000, BF), settings(30, 33)
    tok, lp = run(l, **s)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tok2, lp2 = run(l, **s, stream=side)
    assert (tok == tok2).all() and (lp == lp2).all()
    a = {k: t32(v, torch.int32 if k == "k" else F) for k, v in s.items()}
    out, lps = torch.zeros(33, dtype=torch.int32, device="cuda"), torch.zeros(33, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cce.cce_sample_rows(l, a["t"], a["k"], a["p"], a["mp"], a["u"], out, lps)
    g.replay()
    torch.cuda.synchronize()
    assert (out.cpu().numpy() == tok).all() and (lps.cpu().numpy() == lp).all()
    a["u"].uniform_()
    g.replay()
    check(l, **{**s, "u": a["u"].cpu().numpy()})


def test_logp_is_the_forward_pass_s():
    """The token's logp is cce_forward's for that label."""
    M, D, V = 20, 256, 3000
    g = torch.Generator(device="cuda").manual_seed(3)
    H = torch.randn(M, D, generator=g, device="cuda")
    W = torch.randn(V, D, generator=g, device="cuda") * 0.2
    l = (H.double() @ W.double().T).float()
    tok, lp = run(l, u=np.random.default_rng(1).random(M).astype(np.float32))
    head = cce.Head(w=W, V=V, D=D)
    ws = cce.alloc_workspace(M, cce.CCE_F32, head)
    logp, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    cce.cce_forward(H, head, torch.from_numpy(tok).cuda(), logp, lse, ws=ws)
    torch.cuda.synchronize()
    assert np.abs(logp.cpu().numpy() - lp).max() <= 2e-3  # the head's own tolerance


def test_clusters_that_start_while_the_gpu_is_busy():
    """Rows shared by several CTAs, by list and by search, launched again and
    again beside work that keeps the SMs occupied, so that a cluster's CTAs do
    not begin at the same time: the tokens of a quiet run."""
    jobs = []
    for B, V, dtype in ((10, 20000, F), (3, 70001, BF), (37, 33000, F), (200, 40000, BF)):
        l = logits(B, B, V, dtype, 2.5 if B < 30 else 1.0, B < 30)
        s = {k: t32(v, torch.int32 if k == "k" else F) for k, v in settings(V, B).items()}
        out = [(torch.zeros(B, dtype=torch.int32, device="cuda"), torch.zeros(B, device="cuda"))
               for _ in range(2)]
        jobs.append((l, s, out))

    def launch(stream, which):
        for l, s, out in jobs:
            cce.cce_sample_rows(l, s["t"], s["k"], s["p"], s["mp"], s["u"], *out[which], stream)

    launch(None, 0)
    torch.cuda.synchronize()
    busy, side = torch.cuda.Stream(), torch.cuda.Stream()
    a = torch.randn(2048, 2048, device="cuda", dtype=BF)
    torch.cuda.synchronize()
    for _ in range(30):
        with torch.cuda.stream(busy):
            a @ a
            a.float().sin_()
        launch(side, 1)
        side.synchronize()
        for _, _, (x, y) in jobs:
            assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
            y[0].zero_()
        torch.cuda.current_stream().synchronize()
    torch.cuda.synchronize()


LOWEST = {F: [torch.finfo(BF).min, torch.finfo(F).min, -1e38, -1.2e38],
          BF: [torch.finfo(BF).min, -1e38, -1.2e38]}


@pytest.mark.parametrize("dtype", [F, BF])
@pytest.mark.parametrize("V", [3000, 20000, 140001])
def test_two_masks_in_one_row(V, dtype):
    """Two different very low finite values: their products with log2(e) / T
    are beyond fp32.  In one lane's piece, one segment, two segments of a warp,
    two warps, and over whole stretches, ahead of the live logits and among
    them."""
    places = [((0,), (1,)), ((0,), (300,)), ((0,), (8192 if V > 9000 else 600,)), ((5,), (520,)),
              (range(0, 1000), range(1000, 2000)), (range(0, V - 50, 2), range(1, V - 50, 2))]
    rows = []
    base = logits(V, 1, V, F, 1.0)[0]
    for a in LOWEST[dtype]:
        for b in LOWEST[dtype]:
            if a == b:
                continue
            for pa, pb in places:
                l = base.clone()
                l[list(pa)], l[list(pb)] = a, b
                if pa == (0,):   # nothing live in the first segments
                    l[:512] = a
                    l[list(pb)[0]] = b
                rows.append(l)
    l = torch.stack(rows).to(dtype)
    r = np.random.default_rng(V)
    for i in range(0, l.shape[0], 24):
        x = l[i:i + 24]
        n = x.shape[0]
        for t in (0.0, 0.3, 1.0):
            for p in (0.5, 0.95, 1.0):
                check(x, t=[t] * n, p=[p] * n, u=r.random(n).astype(np.float32))


def test_logits_whose_products_leave_fp32():
    """Maxima of either sign beyond 2.36e38 (times T), alone, repeated, rising
    from segment to segment, and beside infinities."""
    V = 30000
    l = torch.zeros(8, V, device="cuda")
    l[0] = t32(np.linspace(-3.4e38, -2.4e38, V))
    l[1] = t32(np.linspace(-1.6e38, 1.7e38, V))
    l[2] = t32(np.linspace(2e38, 3.4e38, V))
    l[3] = -3e38
    l[3, ::7] = -3.1e38
    l[4] = 3e38
    l[4, ::5] = 2.9e38
    l[5] = l[1]
    l[5, [9, 20000]] = float("inf")
    l[6] = torch.finfo(F).min
    l[6, 1::2] = torch.finfo(BF).min
    l[7, 0] = 3.4e38
    r = np.random.default_rng(8)
    for t in (0.3, 1.0, 5.0, 1e38):
        for p in (1.0, 0.9):
            check(l, t=[t] * 8, p=[p] * 8, u=r.random(8).astype(np.float32))


def test_temperatures_whose_inverse_leaves_fp32():
    """Denormal temperatures with logits of their size, where weights still
    differ, and of ordinary size, where the maximum is alone."""
    V = 30000
    r = np.random.default_rng(12)
    x = np.stack([np.floor(r.random(V) * 4000) * 2.0 ** -149, r.standard_normal(V),
                  -np.floor(r.random(V) * 4000) * 2.0 ** -149, np.zeros(V)])
    l = t32(x)
    for t in (1e-42, 1e-40, 2e-39):
        for p in (1.0, 0.9):
            check(l, t=[t] * 4, p=[p] * 4, u=r.random(4).astype(np.float32))


@pytest.mark.parametrize("V", [3000, 140001])
def test_near_ties_at_the_maximum_of_a_cold_row(V):
    """Many logits a few steps of fp32 below the maximum, at temperatures where
    such a step is worth something: max / T is 1e5 to 1e9, and the fp32 product
    of the two is off by more than the weights differ."""
    r = np.random.default_rng(V)
    B = 24
    x = r.standard_normal((B, V)).astype(np.float32)
    for b in range(B):
        top = np.float32(r.uniform(4, 31) * (1 if b % 2 else -1))
        x[b] = np.minimum(x[b] + min(top, 0) - 8, top - np.float32(1))
        at = r.choice(V, 300, replace=False)
        x[b, at] = top - r.integers(0, 40, 300) * np.spacing(np.abs(top))
    l = t32(x)
    for t in (1e-4, 1e-5, 3e-6, 1e-6, 1e-7):
        for p in (1.0, 0.9, 0.35):
            check(l, t=[t] * B, p=[p] * B, u=r.random(B).astype(np.float32))


def test_logp_of_large_logits():
    """log-softmax at magnitudes where one step of a logit is 0.06 to 8."""
    r = np.random.default_rng(5)
    V = 30000
    rows = []
    for size in (1e6, 4e6, 1.1e7, 2.5e7, 4e7, 1e8):
        for sign in (1, -1):
            top = np.float32(size * r.uniform(0.8, 1.2) * sign)
            rows.append(top - r.integers(0, 12, V) * np.spacing(np.abs(top)))
    l = t32(np.stack(rows))
    n = l.shape[0]
    for t in (0.0, 1.0, 3.0):
        check(l, t=[t] * n, u=r.random(n).astype(np.float32))
        check(l, t=[t] * n, p=[0.6] * n, u=r.random(n).astype(np.float32))


@pytest.mark.parametrize("rise", [2.0, 8.0, 0.3])
def test_logp_of_rows_that_rise_by_segments(rise):
    """150 rows of 2^21 logits, one CTA a row, constant over each 512 and
    rising, so that every segment brings its warp a new maximum (256 times).
    The rows rise by slightly different steps, each over and over.  logp of the
    first rank: the sum's terms, three exponentials and their arguments at
    exponents up to `rise` / ln 2, are off by less than
    (3 2^-22 + 3 2^-24 rise + 10 2^-24) relative, and so is logp absolutely,
    with its own half step."""
    B, V = 150, 1 << 21
    seg = V // 512
    step = np.linspace(0.9, 1.1, B)[:, None] * rise / seg
    x = (step * np.arange(seg)[None]).astype(np.float32)
    l = t32(x).repeat_interleave(512, 1)
    _, lp = run(l, t=[0.0] * B, u=[0.5] * B)
    x = x.astype(np.float64)
    want = -np.log(512 * np.exp(x - x[:, -1:]).sum(1))
    tol = 3 * 2.0 ** -22 + (3 * rise * 1.1 + 10) * 2.0 ** -24 + 2.0 ** -24 * np.abs(want)
    assert (np.abs(lp - want) <= tol).all(), float((np.abs(lp - want) / tol).max())


@pytest.mark.parametrize("V", [7, 3000, 70001])
def test_min_p_around_one_with_equal_maxima(V):
    """min_p = 1 shares the row among the logits at the maximum, above 1 the
    first of them has it alone, with the other settings in force or not."""
    l = logits(V, 12, V, F)
    l[:, [1, 3, V - 1]] = 50.0
    l[8:, [2, 5]] = float("inf")
    mp = [1.0, 1.0 + 2.0 ** -23, 2.0, float("inf")] * 3
    for u in (0.1, 0.5, 0.9):
        tok = check(l, mp=mp, u=[u] * 12)
        assert all(tok[r] == (1 if r < 8 else 2) for r in range(12) if mp[r] > 1)
        check(l, mp=mp, t=[0.5] * 12, k=[20] * 12, p=[0.9] * 12, u=[u] * 12)


@pytest.mark.parametrize("B,V,share", [(5001, 2100, 1.0), (4099, 3000, 0.1), (2048, 9000, 0.5), (40, 40000, 1.0)])
def test_searched_rows_spread_over_a_large_batch(B, V, share):
    """Flat rows (searched) at random places among sharp ones: each gets its
    token once, whichever cluster takes it."""
    r = np.random.default_rng(B)
    flat = r.random(B) < share
    x = np.where(flat[:, None], 0.01, 6.0) * r.standard_normal((B, V))
    l = t32(x)
    u = r.random(B).astype(np.float32)
    check(l, p=[0.9] * B, u=u)


def test_a_million_rows():
    """More rows than the search goes over in a step, none of them left to it."""
    B, V = (1 << 20) + 77, 8
    l = torch.randn(B, V, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    tok, lp = run(l, t=np.zeros(B), u=np.full(B, 0.5))
    assert np.array_equal(tok, l.argmax(1).cpu().numpy())
    want = torch.log_softmax(l.double(), 1).amax(1).cpu().numpy()
    assert (np.abs(lp - want) <= 7e-6 + 2.0 ** -24 * np.abs(want)).all()


def test_maxima_that_rise_by_more_than_weights_hold():
    """Each of a warp's segments outdoes the last one's maximum by 2^100 to
    2^(10^27), at magnitudes where the products with log2(e) / T are rounded by
    as much, up or down."""
    r = np.random.default_rng(14)
    V = 300001
    seg = np.arange(V) // 512
    rise = np.sort(r.random((8, V)), 1)
    rows = [1e30 + 1e24 * seg, -1e30 + 1e24 * seg, 1e12 + 1e6 * seg, 100.0 * seg, 1e6 + 0.0625 * seg,
            1e20 * (1 + seg % 7), 1e9 * r.standard_normal(V)]
    rows += [c * (1 + x * 2.0 ** -14) for c, x in zip((1e30, -1e30, 2e25, 3e20, -7e15, 1e11, 5e8, 1e36), rise)]
    l = t32(np.stack(rows))
    n = l.shape[0]
    for t in (0.0, 1.0, 8.7e-7):
        for p in (1.0, 0.3):
            check(l, t=[t] * n, p=[p] * n, u=r.random(n).astype(np.float32))


def test_logp_far_below_the_maximum_is_rounded_once():
    """Hot rows that take tokens hundreds below the maximum: logp is off by half
    a step, not by another half for the difference."""
    r = np.random.default_rng(15)
    B, V = 64, 20000
    l = t32(-2000 * r.random((B, V)) + r.random((B, 1)) * 50)
    for t in (300.0, 2000.0, 1e30):
        check(l, t=[t] * B, u=r.random(B).astype(np.float32))
