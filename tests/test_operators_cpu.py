"""The operators around a linear layer without a GPU: the reference's own
checks, and every refusal that the library decides on the host (no pointer is
dereferenced, nothing is launched)."""
import os

import numpy as np
import pytest
import torch

import bit_fwht_hadamard_b200 as q
import operators_ref as R

F = 1 << 20                                                  # never dereferenced
BIG = 1 << 40


@pytest.fixture(scope="module", autouse=True)
def _built():
    from bit_fwht_hadamard_b200 import build
    build.build()


# ------------------------------------------------------------------ the reference itself
def test_reference_philox_gives_the_published_vectors():
    path = os.path.join(os.path.dirname(__file__), "golden", "philox_kat.txt")
    n = 0
    for line in open(path):
        w = [t for t in line.split("#")[0].split() if t]
        try:
            v = [int(t, 16) for t in w]
        except ValueError:
            continue
        if len(v) != 10:
            continue
        got = R.philox([np.uint64(t) for t in v[:4]], (v[4], v[5]))
        assert [int(g) for g in got] == v[6:]
        n += 1
    assert n >= 3


def test_reference_slopes_are_the_activations_differences():
    z = torch.linspace(-6, 6, 4001, dtype=torch.float64) + 1e-3
    h = 1e-6
    for name in R.ACTS:
        d = (R.act(z + h, name) - R.act(z - h, name)) / (2 * h)
        # truncation h^2/6 |act'''| and rounding 2^-53 |act| / h
        assert torch.allclose(d, R.slope(z, name), rtol=0, atol=1e-8), name


def test_reference_layernorm_grads_are_differences():
    g = torch.Generator().manual_seed(1)
    x, dy = (torch.randn((5, 12), generator=g, dtype=torch.float64) for _ in range(2))
    gamma, beta = (torch.randn(12, generator=g, dtype=torch.float64) for _ in range(2))
    _, mean, rstd = R.layernorm(x, gamma, beta, 1e-3)
    dx, dg, db = R.layernorm_grads(dy, x, gamma, mean, rstd)

    def loss(x, gamma, beta):
        return float((R.layernorm(x, gamma, beta, 1e-3)[0] * dy).sum())

    h = 1e-6
    for t, d in ((0, dx), (1, dg), (2, db)):
        args = [x, gamma, beta]
        u = torch.randn(args[t].shape, generator=g, dtype=torch.float64)
        lo, hi = list(args), list(args)
        lo[t], hi[t] = args[t] - h * u, args[t] + h * u
        assert abs((loss(*hi) - loss(*lo)) / (2 * h) - float((d * u).sum())) < 1e-7


def test_reference_dropout_keeps_the_right_share():
    k = R.keep((1000, 1000), 0.3, seed=5, step=2)
    assert abs(k.mean() - 0.7) < 4 * np.sqrt(0.21 / 1e6)     # four standard deviations
    assert not np.array_equal(k, R.keep((1000, 1000), 0.3, seed=5, step=3))


# ------------------------------------------------------------------ refusals at the C entry
def _ep(**kw):
    e = q.Epilogue()
    for k, v in kw.items():
        setattr(e, k, v)
    return e


def _gemm(ep=None, M=64, N=64, K=64, fmt=0, out_dt=1, a=F, ts=F, out=F, ws=F, wsb=BIG):
    return q.qfp4_gemm_epilogue(a, F, ts, F, F, ts, M, N, K, fmt, ep, out_dt, out, ws, wsb, None)


def test_gemm_epilogue_refusals():
    assert _gemm(fmt=3) == q.ERR_ARG
    assert _gemm(out_dt=5) == q.ERR_ARG
    assert _gemm(M=-1) == q.ERR_SHAPE
    assert _gemm(K=48) == q.ERR_SHAPE
    assert _gemm(N=66) == q.ERR_SHAPE                        # N % 4, binary32 out
    assert _gemm(N=68, out_dt=0) == q.ERR_SHAPE              # N % 8, bf16 out
    assert _gemm(M=1 << 30) == q.ERR_SHAPE
    assert _gemm(a=None) == q.ERR_ARG
    assert _gemm(out=None) == q.ERR_ARG
    assert _gemm(fmt=q.NVFP4, ts=None) == q.ERR_ARG
    assert _gemm(a=F + 8) == q.ERR_ALIGN
    M, N, K = 4096, 4096, 1024
    need = q.qfp4_gemm_epilogue_workspace_bytes(M, N, K, 0)
    assert need > 0
    assert _gemm(M=M, N=N, K=K, wsb=need - 1) == q.ERR_ARG
    assert _gemm(M=M, N=N, K=K, ws=None) == q.ERR_ARG
    # few tiles, and empty calls, need none
    assert q.qfp4_gemm_epilogue_workspace_bytes(1, 4096, 4096, q.NVFP4) == 0
    assert q.qfp4_gemm_epilogue_workspace_bytes(128, 14336, 4096, q.MXFP8) == 0
    assert q.qfp4_gemm_epilogue_workspace_bytes(0, 4096, 4096, q.NVFP4) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(act=5), q.ERR_ARG), (dict(act=-1), q.ERR_ARG),
    (dict(bias=F, bias_dt=2), q.ERR_ARG), (dict(residual=F, residual_dt=7), q.ERR_ARG),
    (dict(dropout_p=1.0), q.ERR_ARG), (dict(dropout_p=-0.1), q.ERR_ARG), (dict(dropout_p=float("nan")), q.ERR_ARG),
    (dict(bias=F + 2), q.ERR_ALIGN), (dict(residual=F + 4), q.ERR_ALIGN), (dict(preact=F + 8), q.ERR_ALIGN),
    (dict(step=F + 4), q.ERR_ALIGN)])
def test_epilogue_field_refusals(bad, status):
    assert _gemm(_ep(**bad)) == status
    st = q.qfp4_linear_forward_epilogue(F, F, 64, 64, 128, q.NVFP4, 0, _ep(**bad), q.F32, F, F, BIG, None)
    assert st == status


def test_linear_forward_epilogue_refusals():
    L = q.qfp4_linear_forward_epilogue
    e = _ep(act=q.ACT_GELU)
    ws = q.qfp4_linear_forward_workspace_bytes(256, 512, 1024, q.NVFP4)
    assert L(F, F, 256, 512, 1024, 7, 0, e, q.BF16, F, F, BIG, None) == q.ERR_ARG
    assert L(F, F, 256, 512, 1000, q.NVFP4, 0, e, q.BF16, F, F, BIG, None) == q.ERR_SHAPE
    assert L(F, F, 256, 512, 1024, q.MXFP4, 1, e, q.BF16, F, F, BIG, None) == q.ERR_UNSUPPORTED
    assert L(F, F, 256, 512, 1024, q.NVFP4, 0, e, q.BF16, F, F, ws - 1, None) == q.ERR_ARG
    assert L(F, F, 256, 512, 1024, q.NVFP4, 0, e, q.BF16, None, F, BIG, None) == q.ERR_ARG


def test_epilogue_backward_refusals():
    B = q.qfp4_epilogue_backward

    def call(dy=F, z=F, dt=q.F32, M=8, N=8, act=q.ACT_GELU, p=0.1, step=None, dz=F, db=F, ws=F, wsb=BIG):
        return B(dy, z, dt, M, N, act, p, 1, step, dz, db, ws, wsb, None)

    assert call(dt=2) == q.ERR_ARG
    assert call(act=9) == q.ERR_ARG
    assert call(p=1.0) == q.ERR_ARG
    assert call(p=float("nan")) == q.ERR_ARG
    assert call(M=-1) == q.ERR_SHAPE and call(N=1 << 30) == q.ERR_SHAPE
    assert call(dy=None) == q.ERR_ARG and call(dz=None) == q.ERR_ARG
    assert call(z=None) == q.ERR_ARG                         # an activation's slope needs Z
    assert call(dy=F + 2) == q.ERR_ALIGN and call(db=F + 4) == q.ERR_ALIGN and call(step=F + 4) == q.ERR_ALIGN
    need = q.qfp4_epilogue_backward_workspace_bytes(8, 8)
    assert need >= 32
    assert call(wsb=need - 1) == q.ERR_ARG and call(ws=None) == q.ERR_ARG
    assert q.qfp4_epilogue_backward_workspace_bytes(0, 8) == 0


def test_dropout_refusals():
    D = q.qfp4_dropout
    assert D(F, 3, 8, 0.1, 1, None, None, F, None) == q.ERR_ARG
    for p in (1.0, -1e-9, float("nan"), float("inf")):
        assert D(F, q.F32, 8, p, 1, None, None, F, None) == q.ERR_ARG
    assert D(F, q.F32, -1, 0.1, 1, None, None, F, None) == q.ERR_SHAPE
    assert D(F, q.F32, (1 << 38) + 1, 0.1, 1, None, None, F, None) == q.ERR_SHAPE
    assert D(None, q.F32, 8, 0.1, 1, None, None, F, None) == q.ERR_ARG
    assert D(F, q.F32, 8, 0.1, 1, None, None, None, None) == q.ERR_ARG
    assert D(F + 4, q.F32, 8, 0.1, 1, None, None, F, None) == q.ERR_ALIGN
    assert D(F, q.F32, 8, 0.1, 1, F + 4, None, F, None) == q.ERR_ALIGN
    assert D(None, q.F32, 0, 0.1, 1, None, None, None, None) == q.OK        # nothing to do


def test_layernorm_refusals():
    f = q.qfp4_layernorm_forward
    assert f(F, 2, 4, 8, F, F, q.F32, 1e-5, F, F, F, None) == q.ERR_ARG
    assert f(F, q.F32, 4, 8, F, F, 2, 1e-5, F, F, F, None) == q.ERR_ARG
    for eps in (-1e-5, float("nan")):
        assert f(F, q.F32, 4, 8, F, F, q.F32, eps, F, F, F, None) == q.ERR_ARG
    assert f(F, q.F32, 4, 0, F, F, q.F32, 1e-5, F, F, F, None) == q.ERR_SHAPE
    assert f(F, q.F32, -4, 8, F, F, q.F32, 1e-5, F, F, F, None) == q.ERR_SHAPE
    assert f(F, q.F32, 1 << 29, 1 << 12, F, F, q.F32, 1e-5, F, F, F, None) == q.ERR_SHAPE
    assert f(None, q.F32, 4, 8, F, F, q.F32, 1e-5, F, F, F, None) == q.ERR_ARG
    assert f(F, q.F32, 4, 8, F + 4, F, q.F32, 1e-5, F, F, F, None) == q.ERR_ALIGN
    assert f(F, q.F32, 4, 8, F, F, q.F32, 1e-5, F, F + 4, F, None) == q.ERR_ALIGN
    b = q.qfp4_layernorm_backward
    need = q.qfp4_layernorm_backward_workspace_bytes(4, 8)
    assert need >= 2 * 4 * 8

    def call(dy=F, dt=q.F32, M=4, D=8, wdt=q.F32, mean=F, dx=F, dg=F, db=F, ws=F, wsb=BIG):
        return b(dy, F, dt, M, D, F, wdt, mean, F, dx, dg, db, ws, wsb, None)

    assert call(dt=4) == q.ERR_ARG and call(wdt=4) == q.ERR_ARG
    assert call(D=0) == q.ERR_SHAPE and call(M=-1) == q.ERR_SHAPE
    assert call(dx=None, dg=None, db=None) == q.ERR_ARG
    assert call(dy=None) == q.ERR_ARG and call(mean=None) == q.ERR_ARG
    assert call(dy=F + 8) == q.ERR_ALIGN and call(dg=F + 8) == q.ERR_ALIGN
    assert call(wsb=need - 1) == q.ERR_ARG and call(ws=None) == q.ERR_ARG


# ------------------------------------------------------------------ refusals of the torch wrappers
def test_wrappers_refuse_host_tensors():
    x = torch.zeros((64, 64), dtype=torch.bfloat16)
    w = torch.ones(64)
    op = {"codes": torch.zeros((64, 32), dtype=torch.uint8), "scales": torch.zeros((64, 2), dtype=torch.uint8)}
    for call in (lambda: q.gemm_epilogue(op, op, 64, 64, 64, q.MXFP4), lambda: q.linear_forward_epilogue(x, x),
                 lambda: q.epilogue_backward(x, x), lambda: q.dropout(x, 0.1), lambda: q.layernorm_forward(x, w, w),
                 lambda: q.layernorm_backward(x, x, w, w, w)):
        with pytest.raises(ValueError, match="CUDA"):
            call()
