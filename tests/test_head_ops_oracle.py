"""Pins of the oracle of the operators around the head, and the refusals that
need no GPU."""

import ctypes
import subprocess

import numpy as np
import pytest
import torch

from lm_head_cross_flash_b200 import build, cce
from oracle import head_ops as O


@pytest.fixture(scope="module")
def lib():
    build.build()
    return cce.lib()


def test_e4m3_round_matches_the_type():
    """Every e4m3 value is a fixed point, and rounding agrees with torch's
    cast (nearest, ties to even) inside the range."""
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    fin = every[np.isfinite(every)]
    assert np.array_equal(O.e4m3_round(fin), fin)
    r = np.random.default_rng(0)
    v = np.concatenate([r.uniform(-448, 448, 20000), r.uniform(-0.05, 0.05, 20000),
                        (np.sort(fin)[1:] + np.sort(fin)[:-1]) / 2]).astype(np.float32)
    assert np.array_equal(O.e4m3_round(v), torch.from_numpy(v).to(torch.float8_e4m3fn).double().numpy())
    assert O.e4m3_round(1e9) == 448 and O.e4m3_round(-np.inf) == -448


def test_quantised_values_stay_within_half_a_step():
    x = np.random.default_rng(1).standard_normal((7, 300)).astype(np.float32)
    for q, v in ((O.quant_rows(x), O.rows_values), (O.quant_blocks(x), O.blocks_values)):
        got = v(*q)
        m = np.abs(x).max()
        assert (np.abs(got - x) <= np.maximum(np.abs(x) * 2.0 ** -4, m / 448 * 2.0 ** -10) * 1.0001).all()


def test_norm_gradient_is_the_slope():
    r = np.random.default_rng(2)
    x, w, dh = r.standard_normal((3, 50)), r.standard_normal(50), r.standard_normal((3, 50))
    h, rstd = O.norm_forward(x, w, 1e-3)
    dx, dw = O.norm_backward(x * rstd[:, None], rstd, w, dh)
    v, vw, e = r.standard_normal(x.shape), r.standard_normal(50), 1e-6
    f = lambda a, b: (dh * O.norm_forward(x + a * v, w + b * vw, 1e-3)[0]).sum()
    assert abs((f(e, 0) - f(-e, 0)) / (2 * e) - (dx * v).sum()) < 1e-7
    assert abs((f(0, e) - f(0, -e)) / (2 * e) - (dw * vw).sum()) < 1e-7


P = 1 << 20  # an aligned address; refused calls never touch it


def test_quant_refusals(lib):
    for f in (lib.cce_fp8_quant_rows, lib.cce_fp8_quant_blocks):
        bad = [(None, 1, 8, 128, 128, P, 128, P), (P, 1, 0, 128, 128, P, 128, P),
               (P, 1, 8, 0, 128, P, 128, P), (P, 1, 8, 128, 127, P, 128, P),
               (P, 1, 8, 128, 128, None, 128, P), (P, 1, 8, 128, 128, P, 127, P),
               (P, 1, 8, 128, 128, P, 128, None), (P, 7, 8, 128, 128, P, 128, P),
               (P + 1, 1, 8, 128, 128, P, 128, P), (P + 2, 0, 8, 128, 128, P, 128, P),
               (P, 1, 8, 128, 128, P, 128, P + 2)]
        for a in bad:
            assert f(*a, None) == 1, a
        assert f(P, 1, 8, 65537, 65537, P, 65537, P, None) == 2
        assert f(P, 1, (1 << 30) + 1, 8, 8, P, 8, P, None) == 2
    assert lib.cce_fp8_quant_blocks(P, 1, 65535 * 128 + 1, 8, 8, P, 8, P, None) == 2


def test_norm_refusals(lib):
    ok = dict(X=P, xt=1, M=4, D=256, ldx=256, w=P, wt=0, eps=1e-6, H=P, ht=1, ldh=256, H8=None,
              ldh8=0, Hs=None, X8=None, ldx8=0, Xs=None, rstd=None, stream=None)

    def call(**kw):
        return lib.cce_norm_forward(*{**ok, **kw}.values())

    for kw in (dict(X=None), dict(w=None), dict(M=0), dict(D=-1), dict(ldx=255), dict(ldh=255),
               dict(xt=2), dict(wt=-1), dict(ht=5), dict(eps=-1.0), dict(eps=float("nan")),
               dict(H=None), dict(H8=P, ldh8=256), dict(Hs=P), dict(X8=P, ldx8=255, Xs=P),
               dict(rstd=P + 1), dict(X=P + 1), dict(w=P + 2)):
        assert call(**kw) == 1, kw
    assert call(D=16385, ldx=16385, ldh=16385) == 2
    okb = dict(X8=P, ldx8=256, Xs=P, rstd=P, M=4, D=256, w=P, wt=0, dH=P, dht=0, lddh=256, dX=P,
               dxt=1, lddx=256, dW=P, ws=P, n=1 << 20, stream=None)

    def back(**kw):
        return lib.cce_norm_backward(*{**okb, **kw}.values())

    for kw in (dict(X8=None), dict(Xs=None), dict(rstd=None), dict(w=None), dict(dH=None),
               dict(dX=None), dict(ws=None), dict(ws=P + 8), dict(M=0), dict(lddh=1),
               dict(lddx=255), dict(ldx8=0), dict(dht=3), dict(dxt=3), dict(dW=P + 2)):
        assert back(**kw) == 1, kw
    assert back(D=16385, lddh=16385, lddx=16385, ldx8=16385) == 2
    need = lib.cce_norm_backward_workspace_bytes(4, 256)
    assert need > 256 and back(n=need - 1) == 4
    assert lib.cce_norm_backward_workspace_bytes(0, 256) == 0
    assert lib.cce_norm_backward_workspace_bytes(4, 16385) == 0


def test_matmul_refusals(lib):
    ok = dict(A=P, lda=128, SA=P, B=P, ldb=128, SB=P, M=4, N=300, K=128, C=P, ct=1, ldc=300, ws=P,
              n=256, stream=None)

    def call(**kw):
        return lib.cce_fp8_matmul(*{**ok, **kw}.values())

    for kw in (dict(A=None), dict(SA=None), dict(B=None), dict(SB=None), dict(C=None),
               dict(ws=None), dict(A=P + 8), dict(B=P + 8), dict(ws=P + 8), dict(C=P + 1),
               dict(lda=136), dict(ldb=136), dict(lda=112), dict(ldc=299), dict(ct=2), dict(M=0),
               dict(N=0), dict(K=0), dict(SA=P + 2)):
        assert call(**kw) == 1, kw
    assert call(n=255) == 4
    assert call(K=65537, lda=65552, ldb=65552) == 2
    assert call(M=1 << 30, N=1 << 30, ldc=1 << 30) == 2


def test_sampling_oracle_against_closed_forms():
    l = np.log([0.5, 0.2, 0.1, 0.2])
    s = lambda u, k=0, p=1.0, mp=0.0, t=1.0: O.sample_row(l, t, k, p, mp, u)
    assert [s(u)[0] for u in (0.0, 0.49, 0.51, 0.69, 0.71, 0.89, 0.91)] == [0, 0, 1, 1, 3, 3, 2]
    assert abs(s(0.6)[1] - np.log(0.2)) < 1e-12
    assert s(0.99, k=2)[0] == 1 and s(0.99, p=0.6)[0] == 1 and s(0.99, mp=0.45)[0] == 0
    assert s(0.99, k=3, p=0.75)[2].tolist() == [0, 1]   # 0.7 of 0.9 is enough
    assert s(0.7, t=0.0)[0] == 0 and s(0.99, p=0.0)[0] == 0 and s(0.99, mp=5.0)[0] == 0
    assert O.sample_row([-np.inf, np.nan], 1, 0, 1, 0, 0.5)[:2] == (-1, 0.0)
    assert O.sample_row([1.0, np.inf, np.inf], 1, 0, 1, 0, 0.6)[0] == 2


def test_sample_refusals(lib):
    ok = dict(l=P, dt=1, B=4, V=100, ld=100, t=P, k=P, p=P, mp=P, u=P, tok=P, logp=P, stream=None)

    def call(**kw):
        return lib.cce_sample_rows(*{**ok, **kw}.values())

    for kw in (dict(l=None), dict(u=None), dict(tok=None), dict(B=0), dict(V=0), dict(ld=99),
               dict(dt=3), dict(l=P + 1), dict(t=P + 1), dict(k=P + 2), dict(p=P + 1),
               dict(mp=P + 1), dict(u=P + 1), dict(tok=P + 2), dict(logp=P + 1)):
        assert call(**kw) == 1, kw
    assert call(V=(1 << 24) + 1, ld=1 << 25) == 2
    assert call(B=(1 << 24) + 1) == 2


def test_binding_refuses_what_the_library_would_misread():
    cpu = torch.zeros(4, 128)
    with pytest.raises(ValueError, match="CUDA"):
        cce.cce_fp8_quant_rows(cpu, cpu, cpu)
    with pytest.raises(ValueError, match="CUDA"):
        cce.cce_norm_forward(cpu, cpu[0], 1e-6, H=cpu)
    with pytest.raises(ValueError, match="CUDA"):
        cce.cce_norm_backward(cpu, cpu, cpu, cpu, cpu, cpu)
    assert cce.fp8_groups(1) == 1 and cce.fp8_groups(128) == 1 and cce.fp8_groups(129) == 2


def test_min_p_above_one_leaves_the_first_rank():
    """Of several logits at the maximum too: w = 1 is not at least min_p."""
    l = [0.0, 2.0, 2.0, 1.0, 2.0]
    assert O.sample_row(l, 1, 0, 1, 1.0, 0.9)[2].tolist() == [1, 2, 4]
    for mp in (1.0 + 2.0 ** -23, 5.0, np.inf):
        assert O.sample_row(l, 1, 0, 1, mp, 0.9)[2].tolist() == [1]
    assert O.sample_row([1.0, np.inf, np.inf], 1, 0, 1, 2.0, 0.9)[0] == 1


def test_build_checks_the_registers_of_the_hand_over():
    line = ("ptxas info    : Compiling entry function '_ZN3cce15fp8_rows_kernelE14CUtensorMap_stS0_NS_"
            "7Fp8ArgsE' for 'sm_100a'\nptxas info    : Function properties for x\n    0 bytes stack "
            "frame\nptxas info    : Used %d registers, used 16 barriers\n"
            "ptxas info    : Compiling entry function 'y' for 'sm_100a'\n"
            "ptxas info    : Used 168 registers\n")
    build.check_registers(line % 168)
    for bad in (line % 128, line % 255, "", line.replace("fp8_rows", "fp8_few") % 168):
        with pytest.raises(RuntimeError, match="fp8_rows_kernel"):
            build.check_registers(bad)


def test_a_failed_query_is_asked_again(tmp_path):
    """What the driver says of a kernel is kept from the first success on."""
    src = tmp_path / "kept.cpp"
    src.write_text("""
#include "kept.cuh"
int main() {
  static cce::Kept k;
  int asked = 0, v = 0;
  auto fail = [&](int*) { ++asked; return false; };
  auto give = [&](int* n) { ++asked; *n = 168; return true; };
  if (k.get(fail, &v) || k.get(fail, &v) || asked != 2) return 1;
  if (!k.get(give, &v) || v != 168 || asked != 3) return 2;
  v = 0;
  return k.get(fail, &v) && v == 168 && asked == 3 ? 0 : 3;
}
""")
    exe = tmp_path / "kept"
    subprocess.run(["g++", "-std=c++17", "-x", "c++", "-I", build.SRC, "-o", str(exe), str(src)], check=True)
    assert subprocess.run([str(exe)]).returncode == 0


def test_the_norm_and_head_pass_stays_on_one_device(monkeypatch):
    """The head's calls go to the current device and its stream, the norm's to
    the tensors': all three are made with the tensors' device current."""
    now, seen = [torch.device("cuda:0")], []

    class Current:
        def __init__(self, device):
            self.device = torch.device(device)

        def __enter__(self):
            now.append(self.device)

        def __exit__(self, *_):
            now.pop()

    class Any:
        device = torch.device("cuda:1")

        def __getattr__(self, name):
            return None

    monkeypatch.setattr(torch.cuda, "device", Current)
    for f in ("cce_norm_forward", "orpo_head_pass", "cce_norm_backward"):
        monkeypatch.setattr(cce, f, lambda *a, f=f, **k: seen.append((f, now[-1].index)))
    cce.orpo_norm_head_pass(Any(), None, 1e-6, None, None, None, 0.1, "full", 0.0, False, Any(), Any())
    assert seen == [("cce_norm_forward", 1), ("orpo_head_pass", 1), ("cce_norm_backward", 1)]
    assert len(now) == 1


def test_the_norm_s_workspace_holds_a_part_for_each_block(lib):
    """Rows that are not aligned, 257 to 1,024 wide, are taken one by a block:
    as many blocks as rows, up to four on each of 148 SMs (no GPU: the count
    that the library then takes)."""
    for M, D in ((300, 500), (300, 1000), (100, 257), (592, 1023)):
        assert lib.cce_norm_backward_workspace_bytes(M, D) >= 256 + M * D * 4
