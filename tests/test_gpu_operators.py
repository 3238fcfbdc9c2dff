"""The operators around a linear layer on the GPU against their formulas in
binary64 (tests/operators_ref.py), with tolerances counted in roundings:
u = 2^-24 a binary32 operation, finfo.eps / 2 the output's own rounding."""
import numpy as np
import pytest
import torch

import bit_fwht_hadamard_b200 as q
import gpu_util as GU
import operators_ref as R

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
FMT = {"mxfp4": q.MXFP4, "nvfp4": q.NVFP4, "mxfp8": q.MXFP8}
ACT = {n: i for i, n in enumerate(R.ACTS)}


def half_ulp(dt):
    return torch.finfo(dt).eps / 2


def inside(got, want, bound, what):
    got = got.double()
    assert got.shape == want.shape, what
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    err = torch.where(same, torch.zeros_like(want), (got - want).abs())
    bad = ~(err <= bound + 1e-37)
    if bool(bad.any()):
        i = tuple(int(t) for t in bad.nonzero()[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {want.numel()} outside; first at {i}: got {float(got[i])} "
                             f"want {float(want[i])} bound {float(bound[i] if bound.dim() else bound)}")


def normal(shape, seed, std=1.0, dt=F32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dt).cuda()


def step_of(v):
    return torch.tensor([v], dtype=torch.int64, device="cuda")


# ------------------------------------------------------------------ GEMM with an epilogue
def gemm_reference(A, B, fmt, bias, act, p, seed, step, residual):
    """(y, z, bound of y before its rounding, bound of z before its rounding)."""
    a, b = R.values(A, fmt), R.values(B, fmt)
    s, mag = a @ b.T, a.abs() @ b.abs().T
    z = s + (bias.double() if bias is not None else 0.0)
    # the block-scaled product's own bound, then the scale product and one fma
    ez = 1e-5 * mag + 2 * U * (s.abs() + z.abs())
    v = R.act(z, act)
    # slopes stay below 1.13; an activation's evaluation: its exponential and division within 2^-20 (1 + |z|)
    ev = 1.13 * ez + (0.0 if act in ("none", "relu") else 2.0 ** -20 * (1 + z.abs()))
    y = R.drop(v, p, seed, step)
    ey = R.drop(ev, p, seed, step) + 2 * U * y.abs()
    if residual is not None:
        y = y + residual.double()
        ey = ey + U * y.abs()
    return y, z, ey, ez


def check_gemm(M, N, K, fmt, out=BF, bias=None, act="none", preact=False, p=0.0, residual=None, step=None, seed=7):
    A, B = R.random_operand(M, K, FMT[fmt], seed), R.random_operand(N, K, FMT[fmt], seed + 1)
    mag = float(R.values(A, FMT[fmt]).std() * R.values(B, FMT[fmt]).std()) * max(K, 1) ** 0.5 if K else 1.0
    A["scales"], B["scales"] = A["scales"].contiguous(), B["scales"].contiguous()
    bias_t = normal((N,), seed + 2, mag, bias) if bias is not None else None
    res_t = normal((M, N), seed + 3, mag, residual) if residual is not None else None
    y_t = GU.guarded((M, N), out)
    z_t = GU.guarded((M, N), out) if preact else False
    step_t = step_of(step) if step is not None else None
    y, z = q.gemm_epilogue(A, B, M, N, K, FMT[fmt], bias=bias_t, act=ACT[act], want_preact=z_t, dropout_p=p, seed=seed,
                           step=step_t, residual=res_t, out=y_t)
    ry, rz, ey, ez = gemm_reference(A, B, FMT[fmt], bias_t, act, p, seed, step or 0, res_t)
    inside(y, ry, ey + half_ulp(out) * ry.abs() * (1 + 2.0 ** -6), f"y {M}x{N}x{K} {fmt}")
    if preact:
        inside(z, rz, ez + half_ulp(out) * rz.abs() * (1 + 2.0 ** -6), f"preact {M}x{N}x{K} {fmt}")
    assert q.qfp4_last_device_error() == 0
    return y


SIZES = [(1, 8, 32), (1, 4096, 4096), (3, 1000, 2080), (8, 264, 544), (9, 40, 96), (37, 8, 64), (100, 264, 384),
         (128, 512, 4096), (129, 256, 256), (200, 264, 544), (300, 520, 2080), (515, 1032, 160)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("fmt", list(FMT))
def test_gemm_epilogue_all_steps(M, N, K, fmt):
    check_gemm(M, N, K, fmt, BF, bias=BF, act="gelu", preact=True, p=0.25, residual=BF, step=3)


@pytest.mark.parametrize("M,N,K", [(1, 36, 64), (5, 4092, 1056), (16, 300, 9184), (100, 260, 384), (257, 516, 800)])
@pytest.mark.parametrize("fmt", list(FMT))
def test_gemm_epilogue_binary32_out(M, N, K, fmt):
    check_gemm(M, N, K, fmt, F32, bias=F32, act="silu", preact=True, p=0.1, residual=F32, step=(1 << 40) + 5)


@pytest.mark.parametrize("M,N,K", [(1443, 16, 4192), (700, 8, 96), (2264, 136, 1312), (131, 120, 32), (1027, 392, 352)])
@pytest.mark.parametrize("fmt", list(FMT))
def test_gemm_epilogue_narrow_outputs(M, N, K, fmt):
    """Many rows of few columns; scale rows that start on any byte."""
    check_gemm(M, N, K, fmt, BF, bias=F32, act="gelu", preact=True, p=0.25, residual=F32, step=9)
    check_gemm(M, N - 4, K, fmt, F32, bias=BF, residual=BF)


@pytest.mark.parametrize("act", list(ACT))
@pytest.mark.parametrize("M", [2, 70, 300])
def test_gemm_epilogue_activations(act, M):
    check_gemm(M, 264, 512, "nvfp4", F32, bias=BF, act=act, preact=True)


@pytest.mark.parametrize("M", [1, 4, 33, 130])
@pytest.mark.parametrize("opts", [dict(), dict(bias=F32), dict(act="relu"), dict(preact=True), dict(p=0.5),
                                  dict(residual=F32), dict(residual=BF, out=F32), dict(p=0.5, residual=BF)],
                         ids=lambda o: "+".join(o) or "none")
def test_gemm_epilogue_single_steps(M, opts):
    check_gemm(M, 128, 256, "mxfp4", **opts)


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("M", [1, 130])
def test_gemm_epilogue_of_an_empty_sum(fmt, M):
    check_gemm(M, 24, 0, fmt, F32, bias=F32, act="silu", preact=True, p=0.3, residual=BF)


@pytest.mark.parametrize("fmt", list(FMT))
@pytest.mark.parametrize("M", [150, 515])
def test_gemm_epilogue_without_steps_equals_the_gemm(fmt, M):
    """No epilogue: the same kernel steps as q.gemm for more than one row block."""
    N, K = 520, 2080
    A, B = R.random_operand(M, K, FMT[fmt], 3), R.random_operand(N, K, FMT[fmt], 4)
    for dt in (F32, BF):
        y, z = q.gemm_epilogue(A, B, M, N, K, FMT[fmt], out_dtype=dt)
        want = q.gemm(A, B, M, N, K, FMT[fmt], out_dtype=dt)
        assert z is None
        inside(y, want.double(), 2e-5 * (R.values(A, FMT[fmt]).abs() @ R.values(B, FMT[fmt]).abs().T)
               + 2 * half_ulp(dt) * want.double().abs(), "no steps")


@pytest.mark.parametrize("M", [1, 60, 300])
def test_gemm_epilogue_residual_in_place(M):
    N, K = 256, 512
    A, B = R.random_operand(M, K, q.NVFP4, 1), R.random_operand(N, K, q.NVFP4, 2)
    for dt in (BF, F32):
        r = normal((M, N), 3, 100.0, dt)
        want, _ = q.gemm_epilogue(A, B, M, N, K, q.NVFP4, dropout_p=0.2, seed=9, residual=r, out_dtype=dt)
        got, _ = q.gemm_epilogue(A, B, M, N, K, q.NVFP4, dropout_p=0.2, seed=9, residual=r, out=r)
        assert got.data_ptr() == r.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (7, 11008, 4096), (64, 4096, 14336), (2048, 4096, 4096)])
@pytest.mark.parametrize("fmt", list(FMT))
def test_gemm_epilogue_same_bits_again(M, N, K, fmt):
    A, B = R.random_operand(M, K, FMT[fmt], 5), R.random_operand(N, K, FMT[fmt], 6)
    bias, res = normal((N,), 7), normal((M, N), 8, dt=BF)
    ys = [q.gemm_epilogue(A, B, M, N, K, FMT[fmt], bias=bias, act=q.ACT_GELU, dropout_p=0.1, seed=1, residual=res,
                          out_dtype=BF)[0].view(torch.int16) for _ in range(4)]
    assert all(torch.equal(ys[0], y) for y in ys[1:])
    assert q.qfp4_last_device_error() == 0


@pytest.mark.parametrize("M,N,K", [(8192, 11008, 4096), (100, 11008, 4096), (16, 4096, 14336), (128, 14336, 4096)])
def test_gemm_epilogue_full_sizes(M, N, K):
    """Whole outputs at real sizes, so that a wrong tile anywhere shows."""
    check_gemm(M, N, K, "nvfp4", BF, bias=BF, act="gelu", preact=True, p=0.1, residual=BF, step=11)


def test_gemm_epilogue_nan_scale_stays_in_its_row():
    """An E8M0 byte 0xFF makes its row's sums NaN, and no others."""
    M, N, K = 5, 64, 128
    A, B = R.random_operand(M, K, q.MXFP4, 1), R.random_operand(N, K, q.MXFP4, 2)
    A["scales"][2, 1] = 255
    y, _ = q.gemm_epilogue(A, B, M, N, K, q.MXFP4, act=q.ACT_RELU)
    nan = torch.isnan(y).all(1)
    assert nan.tolist() == [False, False, True, False, False]


# ------------------------------------------------------------------ linear layer with an epilogue
@pytest.mark.parametrize("M,N,K", [(1, 264, 384), (100, 264, 384), (256, 512, 1024)])
@pytest.mark.parametrize("mode", ["nvfp4", "nvfp4-four6", "mxfp4"])
def test_linear_forward_epilogue_follows_linear_forward(M, N, K, mode):
    """The epilogue of linear_forward's own binary32 sums."""
    fmt, four6 = FMT[mode[:5]], mode.endswith("four6")
    X, W = normal((M, K), 1, dt=BF), normal((N, K), 2, 0.05, BF)
    bias, res = normal((N,), 3, dt=BF), normal((M, N), 4, dt=BF)
    s = q.linear_forward(X, W, fmt=fmt, four6=four6).double()
    ez = 2e-5 * (X.double().abs() @ W.double().abs().T) * 4 + 2 * U * s.abs()   # the two calls' orders of summation
    y, z = q.linear_forward_epilogue(X, W, fmt=fmt, four6=four6, bias=bias, act=q.ACT_SILU, want_preact=True,
                                     dropout_p=0.3, seed=5, step=step_of(2), residual=res)
    rz = s + bias.double()
    ry = R.drop(R.act(rz, "silu"), 0.3, 5, 2) + res.double()
    inside(z, rz, ez + 2 * U * rz.abs(), "preact")
    inside(y, ry, (1.13 * ez + 2.0 ** -20 * (1 + rz.abs())) / 0.7 + 3 * U * ry.abs(), "y")


# ------------------------------------------------------------------ epilogue backward
def check_epilogue_backward(M, N, dt, act, p, step=None, seed=3, dbias=True):
    dy, z = normal((M, N), seed, dt=dt), normal((M, N), seed + 1, 2.0, dt)
    out = {"dZ": GU.guarded((M, N), dt)}
    if dbias:
        out["dbias"] = GU.guarded((N,), F32)
    dz, db = q.epilogue_backward(dy, z, act=ACT[act], dropout_p=p, seed=seed,
                                 step=step_of(step) if step is not None else None, want_dbias=dbias, out=out)
    d = R.drop(dy.double(), p, seed, step or 0)
    want = d * R.slope(z.double(), act)
    e = 4 * U * want.abs() + (0.0 if act in ("none", "relu") else 2.0 ** -19) * d.abs()   # the slope's evaluation
    inside(dz, want, e + half_ulp(dt) * want.abs() * (1 + 2.0 ** -6), "dz")
    if dbias:
        inside(db, want.sum(0), e.sum(0) + M * U * want.abs().sum(0), "dbias")   # any order of the M terms
    else:
        assert db is None


@pytest.mark.parametrize("M,N", [(1, 1), (1, 8), (3, 5), (17, 1001), (100, 264), (257, 31), (1000, 1030), (2, 20000),
                                 (70000, 3)])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_epilogue_backward_sizes(M, N, dt):
    check_epilogue_backward(M, N, dt, "gelu", 0.3, step=9)


@pytest.mark.parametrize("act", list(ACT))
@pytest.mark.parametrize("p", [0.0, 0.6])
def test_epilogue_backward_activations(act, p):
    check_epilogue_backward(130, 264, F32, act, p)


def test_epilogue_backward_without_dbias():
    check_epilogue_backward(65, 72, BF, "silu", 0.1, dbias=False)


def test_epilogue_backward_without_activation_needs_no_z():
    dy = normal((33, 40), 1)
    dz, db = q.epilogue_backward(dy, dropout_p=0.5, seed=2)
    want = R.drop(dy.double(), 0.5, 2)
    assert torch.equal(dz.double(), want)                    # times two: exact
    inside(db, want.sum(0), 33 * U * want.abs().sum(0), "dbias")


@pytest.mark.parametrize("which", ["dY", "Z"])
@pytest.mark.parametrize("N", [264, 1001])
def test_epilogue_backward_in_place(which, N):
    dy, z = normal((50, N), 1, dt=BF), normal((50, N), 2, dt=BF)
    want, wb = q.epilogue_backward(dy, z, act=q.ACT_GELU_TANH, dropout_p=0.2, seed=4)
    t = dy if which == "dY" else z
    got, gb = q.epilogue_backward(dy, z, act=q.ACT_GELU_TANH, dropout_p=0.2, seed=4, out={"dZ": t})
    assert torch.equal(got, want) and torch.equal(gb, wb)


@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_epilogue_backward_extreme_z(dt):
    """Saturated activations: finite slopes 0 or 1, and a NaN stays one."""
    z = torch.tensor([[0.0, -0.0, 1e30, -1e30, 80.0, -80.0, 3e38, -3e38, float("nan"), 1e-30, -30.0, 30.0]], dtype=dt,
                     device="cuda")
    dy = torch.ones_like(z)
    for name in ("gelu", "gelu_tanh", "silu"):
        got, _ = q.epilogue_backward(dy, z, act=ACT[name])
        want = torch.tensor([[.5, .5, 1, 0, 1, 0, 1, 0, float("nan"), .5, 0, 1]], device="cuda", dtype=torch.float64)
        inside(got, want, 2.0 ** -19 * torch.ones_like(want), name)
    got, _ = q.epilogue_backward(dy, z, act=q.ACT_RELU)
    assert got[0, :8].tolist() == [0, 0, 1, 0, 1, 0, 1, 0] and float(got[0, 9]) == 1


@pytest.mark.parametrize("act", list(ACT))
def test_epilogue_gradient_against_differences(act):
    """dz and dbias as directional differences of the formula in binary64."""
    M, N = 12, 40
    dy, z = normal((M, N), 1), normal((M, N), 2, 1.5)
    z = torch.where(z.abs() < 1e-3, torch.full_like(z, 0.1), z)                  # away from relu's corner
    dz, db = q.epilogue_backward(dy, z, act=ACT[act], dropout_p=0.4, seed=8)
    h = 1e-5

    def loss(zz):
        return (R.drop(R.act(zz, act), 0.4, 8) * dy.double()).sum()

    u, b = normal((M, N), 3).double(), normal((N,), 4).double()
    for d, grad in ((u, dz), (b.expand(M, N), db.expand(M, N) / M)):
        diff = float((loss(z.double() + h * d) - loss(z.double() - h * d)) / (2 * h))
        have = float((grad.double() * d).sum())
        # evaluation 2^-19 a term, the difference's h^2 |f'''| (third derivatives below 4) and 2^-50 / h
        assert abs(diff - have) <= 2.0 ** -19 * float((dy.double() * d).abs().sum()) / 0.6 + 1e-6


# ------------------------------------------------------------------ dropout
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 7, 8, 9, 4095, 4097, 515 * 1001, 1 << 20])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("res", [False, True], ids=["alone", "residual"])
def test_dropout(n, dt, res):
    x, r = normal((n,), 1, dt=dt), normal((n,), 2, 3.0, dt) if res else None
    p, seed, step = 0.3, (1 << 63) + 12345, 77
    y = q.dropout(x, p, seed=seed, step=step_of(step), residual=r, out=GU.guarded((n,), dt))
    want = R.drop(x.double(), p, seed, step)
    e = 2 * U * want.abs()                                    # 1 / (1 - p) and the product
    if res:
        want = want + r.double()
        e = e + U * want.abs()
    inside(y, want, e + half_ulp(dt) * want.abs() * (1 + 2.0 ** -6), "dropout")


def test_dropout_keeps_everything_at_zero_and_little_near_one():
    x = normal((1000,), 1)
    assert torch.equal(q.dropout(x, 0.0, seed=3), x)
    y = q.dropout(x, 1 - 2.0 ** -10, seed=3)
    assert torch.equal(y, R.drop(x.double(), 1 - 2.0 ** -10, 3).float())         # times 1024: exact


def test_dropout_drops_infinities_and_nan():
    x = torch.full((4096,), float("inf"), device="cuda")
    x[::2] = float("nan")
    y = q.dropout(x, 0.5, seed=1)
    k = torch.from_numpy(R.keep((4096,), 0.5, 1)).cuda()
    assert bool((y[~k] == 0).all()) and not bool(torch.isfinite(y[k]).any())


def test_dropout_backward_is_the_same_call_and_in_place():
    x = normal((33, 1001), 1, dt=BF)
    y = q.dropout(x, 0.2, seed=5)
    g = torch.ones_like(x)
    d = q.dropout(g, 0.2, seed=5, out=g)
    assert d.data_ptr() == g.data_ptr()
    assert torch.equal((d != 0), torch.from_numpy(R.keep((33, 1001), 0.2, 5)).cuda())
    assert torch.equal((d != 0) & (x != 0), y != 0)


def test_dropout_empty():
    assert q.dropout(torch.empty((0, 5), device="cuda"), 0.1).shape == (0, 5)


def test_epilogue_and_dropout_draw_the_same_mask():
    """One generator: the GEMM's dropout, its backward and q.dropout agree."""
    for M in (3, 40, 200):
        N = 264
        A, B = R.random_operand(M, 0, q.MXFP4, 1), R.random_operand(N, 0, q.MXFP4, 2)
        one = torch.ones((N,), device="cuda")
        y, _ = q.gemm_epilogue(A, B, M, N, 0, q.MXFP4, bias=one, dropout_p=0.5, seed=6, step=step_of(4))
        want = q.dropout(torch.ones((M, N), device="cuda"), 0.5, seed=6, step=step_of(4))
        back, _ = q.epilogue_backward(torch.ones((M, N), device="cuda"), dropout_p=0.5, seed=6, step=step_of(4))
        assert torch.equal(y, want) and torch.equal(back, want)


# ------------------------------------------------------------------ layer norm
def norm_bounds(x, D):
    """(relative roundings of a row's sum, bound of the mean): a thread adds
    at most D / 256 + 48 terms one after the other, and a tree of ten levels
    joins the threads."""
    L = D / 256 + 64
    return L, L * U * x.abs().mean(-1)


def norm_input(M, D, dt, seed=1):
    return (normal((M, D), seed, 1.5) + normal((M, 1), seed + 1)).to(dt)


def check_layernorm(M, D, dt, wdt, eps=1e-5, params=True, x=None, stats=True):
    x = norm_input(M, D, dt) if x is None else x
    g = (1 + normal((D,), 3, 0.3)).to(wdt) if params else None
    b = normal((D,), 4, 0.3, wdt) if params else None
    out = {"y": GU.guarded((M, D), dt)}
    if stats:
        out |= {"mean": GU.guarded((M,), F32), "rstd": GU.guarded((M,), F32)}
    y, mean, rstd = q.layernorm_forward(x, g, b, eps=eps, want_stats=stats, out=out)
    eps32 = float(np.float32(eps))
    xd, gd = x.double(), g.double() if params else torch.ones(D, device="cuda", dtype=torch.float64)
    ry, rm, rr = R.layernorm(xd, g.double() if params else None, b.double() if params else None, eps32)
    L, em = norm_bounds(xd, D)
    er = (L + 8) * U + 2 * em * em * rr * rr                  # of rstd, relative
    if stats:
        inside(mean, rm, em + U * rm.abs(), "mean")
        inside(rstd, rr, er * rr, "rstd")
    xh = (xd - rm[:, None]) * rr[:, None]
    ey = gd.abs() * (em * rr)[:, None] + (gd * xh).abs() * (er[:, None] + 6 * U) + 2 * U * ry.abs()
    inside(y, ry, ey + half_ulp(dt) * ry.abs() * (1 + 2.0 ** -6), f"y {M}x{D}")


NORM_SIZES = [(1, 1), (5, 2), (3, 7), (4, 32), (9, 100), (2, 255), (33, 256), (4, 768), (7, 1000), (3, 1001),
              (5, 1024), (6, 2040), (2, 4096), (3, 5003), (4, 8192), (2, 16384), (2, 16385), (1, 40000), (3, 65536),
              (5000, 24), (700, 264)]


@pytest.mark.parametrize("M,D", NORM_SIZES)
@pytest.mark.parametrize("dt,wdt", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)],
                         ids=["bf16", "bf16-f32", "f32", "f32-bf16"])
def test_layernorm_forward(M, D, dt, wdt):
    check_layernorm(M, D, dt, wdt)


def test_layernorm_forward_without_parameters_or_statistics():
    check_layernorm(9, 520, BF, BF, params=False, stats=False)
    check_layernorm(9, 4099, F32, F32, params=False, stats=False)


@pytest.mark.parametrize("D", [64, 1001, 4096])
def test_layernorm_forward_far_from_zero(D):
    """A mean a thousand times the deviation: the second pass subtracts it first."""
    x = (1000 + normal((7, D), 5)).contiguous()
    check_layernorm(7, D, F32, F32, x=x)


def test_layernorm_of_constant_rows():
    for D in (8, 333, 4096):
        x = torch.full((3, D), 2.5, device="cuda")
        y, mean, rstd = q.layernorm_forward(x, eps=1e-5)
        assert bool((y == 0).all()) and bool((mean == 2.5).all())
        assert torch.allclose(rstd.double(), torch.full((3,), 1e-5 ** -0.5, device="cuda", dtype=torch.float64),
                              rtol=8 * U, atol=0)


def test_layernorm_in_place_and_nan_rows():
    for D in (100, 4096, 20000):
        x = norm_input(6, D, F32)
        x[2, 5] = float("nan")
        x[4, 7] = float("inf")
        want, _, _ = q.layernorm_forward(x)
        got, _, _ = q.layernorm_forward(x, out={"y": x})
        assert torch.isnan(want).all(1).tolist() == [False, False, True, False, True, False]
        assert torch.equal(torch.nan_to_num(got), torch.nan_to_num(want))


def check_layernorm_backward(M, D, dt, wdt, params=True):
    x, dy = norm_input(M, D, dt), normal((M, D), 7, dt=dt)
    g = (1 + normal((D,), 3, 0.3)).to(wdt) if params else None
    _, rm, rr = R.layernorm(x.double(), None, None, 1e-5)
    mean, rstd = rm.float(), rr.float()
    out = {"dx": GU.guarded((M, D), dt), "dgamma": GU.guarded((D,), F32), "dbeta": GU.guarded((D,), F32)}
    dx, dg, db = q.layernorm_backward(dy, x, g, mean, rstd, out=out)
    gd = g.double() if params else None
    wx, wg, wb = R.layernorm_grads(dy.double(), x.double(), gd, mean.double(), rstd.double())
    L, _ = norm_bounds(x.double(), D)
    # xhat: x - mean rounds relative to the two, then the product with rstd
    ax = (x.double().abs() + mean.double().abs()[:, None]) * rstd.double()[:, None]
    exh = 3 * U * ax
    xh = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    gg = dy.double() * (gd if params else 1.0)
    e1 = (L + 2) * U * gg.abs().mean(-1, keepdim=True)
    e2 = (L + 2) * U * (gg * xh).abs().mean(-1, keepdim=True) + (gg.abs() * exh).mean(-1, keepdim=True)
    c2 = (gg * xh).mean(-1, keepdim=True).abs()
    ex = rstd.double()[:, None] * (3 * U * gg.abs() + e1 + xh.abs() * (e2 + 4 * U * c2) + exh * c2
                                   + 4 * U * gg.abs().mean(-1, keepdim=True))
    inside(dx, wx, ex + (2 * U + half_ulp(dt) * (1 + 2.0 ** -6)) * wx.abs(), f"dx {M}x{D}")
    inside(dg, wg, (M + 4) * U * (dy.double() * xh).abs().sum(0) + (dy.double().abs() * exh).sum(0), f"dgamma {M}x{D}")
    inside(db, wb, M * U * dy.double().abs().sum(0), f"dbeta {M}x{D}")


@pytest.mark.parametrize("M,D", NORM_SIZES + [(70000, 3), (300, 4096), (1000, 1030)])
@pytest.mark.parametrize("dt,wdt", [(BF, BF), (BF, F32), (F32, F32)], ids=["bf16", "bf16-f32", "f32"])
def test_layernorm_backward(M, D, dt, wdt):
    check_layernorm_backward(M, D, dt, wdt)


def test_layernorm_backward_without_parameters_and_in_parts():
    check_layernorm_backward(40, 520, BF, BF, params=False)
    for M, D in ((40, 520), (40, 1001), (300, 4096), (3, 20000)):
        x, dy = norm_input(M, D, F32), normal((M, D), 2)
        g = 1 + normal((D,), 3, 0.3)
        _, mean, rstd = q.layernorm_forward(x, g)
        dx, dg, db = q.layernorm_backward(dy, x, g, mean, rstd)
        only, none, none2 = q.layernorm_backward(dy, x, g, mean, rstd, want_dw=False)
        assert none is None and none2 is None and torch.equal(only, dx)
        nodx, dg2, db2 = q.layernorm_backward(dy, x, g, mean, rstd, want_dx=False)
        assert nodx is None and torch.equal(dg2, dg) and torch.equal(db2, db)
        _, dg3, no = q.layernorm_backward(dy, x, g, mean, rstd, want_dw=False,
                                          out={"dgamma": torch.empty_like(dg)})
        assert no is None and torch.equal(dg3, dg)
        over, dg4, db4 = q.layernorm_backward(dy, x, g, mean, rstd, out={"dx": dy})     # dx over dy
        assert torch.equal(over, dx) and torch.equal(dg4, dg) and torch.equal(db4, db)


def test_layernorm_gradient_against_differences():
    M, D = 6, 48
    x, dy = norm_input(M, D, F32), normal((M, D), 7)
    g, b = 1 + normal((D,), 3, 0.3), normal((D,), 4)
    _, mean, rstd = q.layernorm_forward(x, g, b)
    grads = q.layernorm_backward(dy, x, g, mean, rstd)
    h, eps32 = 1e-5, float(np.float32(1e-5))
    args = [x.double(), g.double(), b.double()]
    for t, grad in enumerate(grads):
        u = normal(args[t].shape, 20 + t).double()
        lo, hi = list(args), list(args)
        lo[t], hi[t] = args[t] - h * u, args[t] + h * u
        diff = float(((R.layernorm(*hi, eps32)[0] - R.layernorm(*lo, eps32)[0]) * dy.double()).sum() / (2 * h))
        # 48-term sums and products in binary32: below 2^-16 of the terms; h^2 and 2^-50 / h of the difference
        assert abs(diff - float((grad.double() * u).sum())) <= 2.0 ** -16 * float((grad.double() * u).abs().sum()) + 1e-5


def test_layernorm_empty():
    y, mean, rstd = q.layernorm_forward(torch.empty((0, 64), device="cuda"))
    assert y.shape == (0, 64) and mean.shape == (0,)
    z = torch.empty((0,), device="cuda")
    dx, dg, db = q.layernorm_backward(y, y, torch.ones(64, device="cuda"), z, z)
    assert dx.shape == (0, 64) and bool((dg == 0).all()) and bool((db == 0).all())
    dz, db = q.epilogue_backward(torch.empty((0, 16), device="cuda"))
    assert bool((db == 0).all())


# ------------------------------------------------------------------ streams, graphs, a block of them
def test_operators_on_another_stream():
    s = torch.cuda.Stream()
    x = normal((300, 1024), 1, dt=BF)
    g = normal((1024,), 2, dt=BF)
    A, B = R.random_operand(300, 512, q.NVFP4, 1), R.random_operand(256, 512, q.NVFP4, 2)
    want = [q.layernorm_forward(x, g)[0], q.dropout(x, 0.2, seed=1), q.gemm_epilogue(A, B, 300, 256, 512, q.NVFP4)[0],
            *q.epilogue_backward(x, x, act=q.ACT_GELU)]
    s.wait_stream(torch.cuda.current_stream())
    got = [q.layernorm_forward(x, g, stream=s)[0], q.dropout(x, 0.2, seed=1, stream=s),
           q.gemm_epilogue(A, B, 300, 256, 512, q.NVFP4, stream=s)[0],
           *q.epilogue_backward(x, x, act=q.ACT_GELU, stream=s)]
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("fmt,M,N,K", [("nvfp4", 4, 8960, 1024), ("mxfp8", 20, 4480, 1024), ("mxfp4", 2, 2304, 2048)])
def test_gemm_epilogue_of_few_rows_on_two_streams_at_once(fmt, M, N, K):
    """Clusters of two calls that run together: with so short a K two CTAs
    would fit on an SM, and each takes the whole tensor memory."""
    calls = []
    for seed in (1, 11):
        A, B = R.random_operand(M, K, FMT[fmt], seed), R.random_operand(N, K, FMT[fmt], seed + 1)
        bias = normal((N,), seed + 2)
        calls.append(lambda A=A, B=B, bias=bias, **kw: q.gemm_epilogue(A, B, M, N, K, FMT[fmt], bias=bias,
                                                                       act=q.ACT_SILU, **kw)[0])
    want = [f() for f in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[], []]
    for _ in range(40):
        for k in (0, 1):
            got[k].append(calls[k](stream=streams[k]))
    torch.cuda.synchronize()
    for k in (0, 1):
        assert all(torch.equal(g, want[k]) for g in got[k])
    assert q.qfp4_last_device_error() == 0


def test_graph_replays_draw_new_masks():
    """The step counter is read when the kernel runs: each replay has its own mask."""
    x = torch.ones((64, 256), device="cuda")
    step = step_of(0)
    y = torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        q.dropout(x, 0.5, seed=3, step=step, out=y)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.dropout(x, 0.5, seed=3, step=step, out=y)
        step.add_(1)
    step.zero_()
    for k in range(3):
        graph.replay()
        assert torch.equal(y.double(), R.drop(x.double(), 0.5, 3, k))


def test_two_captured_graphs_with_their_own_workspaces():
    """Each capture takes its workspaces from its own pool: replays in turn and
    overlapping give what eager calls give."""
    def make(seed, M, act):
        A, B = R.random_operand(M, 512, q.NVFP4, seed), R.random_operand(256, 512, q.NVFP4, seed + 1)
        x, dy = norm_input(M, 256, F32, seed), normal((M, 256), seed + 2)
        g = normal((256,), seed + 3)

        def work():
            y, z = q.gemm_epilogue(A, B, M, 256, 512, q.NVFP4, act=act, want_preact=True, dropout_p=0.1, seed=seed)
            dz, db = q.epilogue_backward(y, z, act=act, dropout_p=0.1, seed=seed)
            n, mean, rstd = q.layernorm_forward(x, g)
            return [y, z, dz, db, n, *q.layernorm_backward(dy, x, g, mean, rstd)]
        return work

    works = [make(1, 300, q.ACT_GELU), make(50, 40, q.ACT_SILU), make(90, 3, q.ACT_RELU)]
    want = [w() for w in works]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for w in works:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(w())
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(3):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, outs):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_refusals_of_the_wrappers_on_cuda_tensors():
    x = normal((8, 64), 1)
    w = normal((64,), 2)
    A, B = R.random_operand(8, 64, q.NVFP4, 1), R.random_operand(16, 64, q.NVFP4, 2)
    with pytest.raises(ValueError, match="shape"):
        q.gemm_epilogue(A, B, 8, 24, 64, q.NVFP4)
    with pytest.raises(ValueError, match="bias"):
        q.gemm_epilogue(A, B, 8, 16, 64, q.NVFP4, bias=normal((8,), 1))
    with pytest.raises(ValueError, match="residual"):
        q.gemm_epilogue(A, B, 8, 16, 64, q.NVFP4, residual=normal((16, 8), 1))
    with pytest.raises(TypeError):
        q.gemm_epilogue(A, B, 8, 16, 64, q.NVFP4, out_dtype=torch.float16)
    with pytest.raises(TypeError):
        q.gemm_epilogue(A, B, 8, 16, 64, q.NVFP4, step=torch.zeros(1, device="cuda"))
    with pytest.raises(q.QFP4Error):
        q.gemm_epilogue(A, B, 8, 16, 64, q.NVFP4, dropout_p=1.0)
    with pytest.raises(ValueError, match="workspace"):
        q.epilogue_backward(x, workspace=torch.empty(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="workspace"):
        q.layernorm_backward(x, x, w, x[:, 0].contiguous(), x[:, 1].contiguous(),
                             workspace=torch.empty((4, 4096), device="cuda").T)
    with pytest.raises(q.QFP4Error):                          # too small
        q.epilogue_backward(x, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        q.dropout(x.T, 0.1)
    with pytest.raises(TypeError):
        q.dropout(x.half(), 0.1)
    with pytest.raises(ValueError, match="gamma"):
        q.layernorm_forward(x, normal((63,), 1))
    with pytest.raises(TypeError):
        q.layernorm_forward(x, w, w.bfloat16())
    with pytest.raises(TypeError):
        q.epilogue_backward(x, x.bfloat16(), act=q.ACT_GELU)
    with pytest.raises(q.QFP4Error):
        q.epilogue_backward(x, None, act=q.ACT_GELU)
    with pytest.raises(q.QFP4Error):                          # a view off 16 bytes
        q.dropout(normal((65,), 1)[1:], 0.1)


def test_a_transformer_block_forward_and_backward():
    """Norm, up projection (bias, GELU), down projection (bias, dropout,
    residual) and the way back, as a training step calls them, against the
    same chain with the epilogues and norms in binary64 around the library's
    own quantized products."""
    M, D, H = 256, 512, 1024
    x = normal((M, D), 1, dt=BF)
    g, b = (1 + normal((D,), 2, 0.2)).to(BF), normal((D,), 3, 0.2, BF)
    W1, W2 = normal((H, D), 4, 0.05, BF), normal((D, H), 5, 0.03, BF)
    b1, b2 = normal((H,), 6, 0.2, BF), normal((D,), 7, 0.2, BF)
    p, seed, step = 0.1, 21, step_of(5)
    n, mean, rstd = q.layernorm_forward(x, g, b)
    h, z1 = q.linear_forward_epilogue(n, W1, bias=b1, act=q.ACT_GELU, want_preact=True, out_dtype=BF)
    y, _ = q.linear_forward_epilogue(h, W2, bias=b2, dropout_p=p, seed=seed, step=step, residual=x, out_dtype=BF)
    gy = normal((M, D), 8, 0.1, BF)
    d2, db2 = q.epilogue_backward(gy, dropout_p=p, seed=seed, step=step)
    dh, dW2 = q.linear_backward(d2, h, W2, seed=1, out_dtype=BF)
    d1, db1 = q.epilogue_backward(dh, z1, act=q.ACT_GELU)
    dn, dW1 = q.linear_backward(d1, n, W1, seed=2, out_dtype=BF)
    dx, dg, dbeta = q.layernorm_backward(dn, x, g, mean, rstd)
    dx = dx + gy                                              # the residual's own gradient
    # each link against binary64 on the link's own inputs
    e = half_ulp(BF) * (1 + 2.0 ** -6)
    rn, rm, rr = R.layernorm(x.double(), g.double(), b.double(), float(np.float32(1e-5)))
    inside(n, rn, (e + 2.0 ** -16) * rn.abs() + 2.0 ** -16, "norm")
    s1 = q.linear_forward(n, W1).double() + b1.double()
    t1 = 2.0 ** -16 * (1 + s1.abs())
    inside(z1, s1, e * s1.abs() + t1, "up, before the GELU")
    inside(h, R.act(s1, "gelu"), e * R.act(s1, "gelu").abs() + 2 * t1, "up")
    s2 = q.linear_forward(h, W2).double() + b2.double()
    ry = R.drop(s2, p, seed, 5) + x.double()
    inside(y, ry, e * ry.abs() + 2.0 ** -16 * (1 + s2.abs()), "down")
    inside(d2, R.drop(gy.double(), p, seed, 5), 2 * e * R.drop(gy.double(), p, seed, 5).abs(), "dropout's gradient")
    r1 = dh.double() * R.slope(z1.double(), "gelu")
    inside(d1, r1, e * r1.abs() + 2.0 ** -18 * dh.double().abs(), "GELU's gradient")
    inside(db1, r1.sum(0), 2.0 ** -15 * dh.double().abs().sum(0), "bias gradient")
    rx, rg, rb = R.layernorm_grads(dn.double(), x.double(), g.double(), mean.double(), rstd.double())
    inside(dg, rg, 2.0 ** -15 * (dn.double().abs() * 4).sum(0), "gamma")
    inside(dbeta, rb, 2.0 ** -15 * dn.double().abs().sum(0), "beta")
    rx = rx + gy.double()
    inside(dx, rx, 3 * e * (rx.abs() + gy.double().abs()) + 2.0 ** -15 * rr[:, None], "dx")
    assert dW1.shape == W1.shape and dW2.shape == W2.shape
    assert all(bool(torch.isfinite(t).all()) for t in (dW1, dW2, db1, db2))


# ------------------------------------------------------------------ offsets past 31 and 32 bits
def test_dropout_past_32_bits():
    """2^32 + 12 elements: every index in 64 bits, the counters' low words up to 2^30."""
    n = (1 << 32) + 12
    x = torch.ones((n,), dtype=BF, device="cuda")
    y = q.dropout(x, 0.5, seed=4, step=step_of(3))
    for start in (0, (1 << 31) - 8, (1 << 32) - 8):
        k = torch.from_numpy(R.keep_range(start, 20, 0.5, 4, 3)).cuda()
        assert torch.equal(y[start:start + 20] == 2, k) and torch.equal(y[start:start + 20] == 0, ~k)
    kept = sum(int((c == 2).sum()) for c in y.split(1 << 28))
    assert abs(kept - n / 2) < 6 * (n / 4) ** 0.5             # six standard deviations


@pytest.mark.parametrize("D", [2056, 2051])
def test_row_operators_past_31_bits(D):
    """More than 2^31 elements: the last rows equal the same rows alone."""
    M = (1 << 31) // D + 9
    tail = normal((16, D), 1, dt=BF)
    x = torch.empty((M, D), dtype=BF, device="cuda")
    x[:-16].fill_(0.25)
    x[-16:] = tail
    g = 1 + normal((D,), 2, 0.3)
    y, mean, rstd = q.layernorm_forward(x, g)
    wy, wm, wr = R.layernorm(tail.double(), g.double(), None, float(np.float32(1e-5)))
    inside(y[-16:], wy, 2.0 ** -8 * wy.abs() + 2.0 ** -16, "y")
    inside(mean[-16:], wm, torch.full_like(wm, 2.0 ** -16), "mean")
    del y
    dx, dg, db = q.layernorm_backward(x, x, g, mean, rstd)
    # the constant rows have xhat = 0 to rounding (their rstd is 1e-5^-1/2)
    wx, wg, wb = R.layernorm_grads(tail.double(), tail.double(), g.double(), mean[-16:].double(), rstd[-16:].double())
    inside(dx[-16:], wx, 2.0 ** -8 * wx.abs() + 2.0 ** -14, "dx")
    inside(db, wb + 0.25 * (M - 16), torch.full_like(wb, M * U * 0.25 * M), "dbeta")
    del dx
    dz, dbias = q.epilogue_backward(x, x, act=q.ACT_SILU, dropout_p=0.5, seed=3)
    first = (M - 16) * D // 4 * 4
    k = torch.from_numpy(R.keep_range(first, M * D - first, 0.5, 3)).cuda()[(M - 16) * D - first:].view(16, D)
    want = torch.where(k, 2 * tail.double() * R.slope(tail.double(), "silu"), torch.zeros((16, D), device="cuda").double())
    inside(dz[-16:], want, 2.0 ** -8 * want.abs() + 2.0 ** -18 * tail.double().abs(), "dz")


def test_gemm_epilogue_past_31_bits():
    """An output of more than 2^31 elements: its last rows equal a small call's."""
    M, N, K = 65552, 32776, 32
    A, B = R.random_operand(M, K, q.MXFP4, 1), R.random_operand(N, K, q.MXFP4, 2)
    y, _ = q.gemm_epilogue(A, B, M, N, K, q.MXFP4, act=q.ACT_RELU, out_dtype=BF)
    t = {k: v[-200:].clone() for k, v in A.items()}
    want, _ = q.gemm_epilogue(t, B, 200, N, K, q.MXFP4, act=q.ACT_RELU, out_dtype=BF)
    assert torch.equal(y[-200:], want)                        # sums of one k-tile are exact


def test_layernorm_ring_of_many_rows_is_the_same_again():
    """Rows through the copies' ring many times over: the same bits each time."""
    for M, D, dt in ((5000, 4096, BF), (3001, 1024, BF), (2000, 8192, F32), (999, 16384, BF)):
        x, dy = norm_input(M, D, dt), normal((M, D), 2, dt=dt)
        g = 1 + normal((D,), 3, 0.3)
        _, mean, rstd = q.layernorm_forward(x, g)
        first = q.layernorm_backward(dy, x, g, mean, rstd)
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(first, q.layernorm_backward(dy, x, g, mean, rstd)))
        wx, wg, wb = R.layernorm_grads(dy.double(), x.double(), g.double(), mean.double(), rstd.double())
        assert float((first[1].double() - wg).norm() / wg.norm()) < 1e-6
        assert float((first[2].double() - wb).norm() / wb.norm()) < 1e-6
    assert q.qfp4_last_device_error() == 0
