"""Each kernel variant behind the operators around a linear layer, at sizes
that its dispatch rule gives to it: the CTA-pair GEMM's epilogue, the few-row
GEMM's column epilogue, layer norm of many rows, gradients of long rows.
Bounds as in test_gpu_operators.py."""
import pytest
import torch

import bit_fwht_hadamard_b200 as q
import operators_ref as R
import test_gpu_operators as T

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
FMT = T.FMT


def pair_runs(M, N, K, fmt):
    """The CTA-pair kernel is the one with a workspace (for the rearranged scales)."""
    return q.qfp4_gemm_epilogue_workspace_bytes(M, N, K, FMT[fmt]) > 0


# ------------------------------------------------------------------ the CTA-pair kernel's epilogue
# more than 148 tiles of 128 x 128, ragged in M, N and K; 1600 columns start every row on 32 bytes, the others do not
@pytest.mark.parametrize("M,N,K", [(1667, 1544, 160), (1300, 2056, 96), (1601, 1600, 1056), (2049, 1288, 2080)])
@pytest.mark.parametrize("fmt", list(FMT))
def test_pair_epilogue_all_steps(M, N, K, fmt):
    assert pair_runs(M, N, K, fmt)
    T.check_gemm(M, N, K, fmt, BF, bias=BF, act="gelu", preact=True, p=0.25, residual=BF, step=3)


@pytest.mark.parametrize("M,N,K", [(2060, 1292, 2080), (1667, 1540, 160), (1601, 1600, 1056)])
@pytest.mark.parametrize("fmt", list(FMT))
def test_pair_epilogue_binary32_out(M, N, K, fmt):
    assert pair_runs(M, N, K, fmt)
    T.check_gemm(M, N, K, fmt, F32, bias=F32, act="silu", preact=True, p=0.1, residual=F32, step=(1 << 40) + 5)


@pytest.mark.parametrize("act", list(T.ACT))
@pytest.mark.parametrize("out,bias,residual", [(BF, F32, F32), (F32, BF, BF), (BF, None, BF)],
                         ids=["bf16-f32", "f32-bf16", "bf16-bf16"])
def test_pair_epilogue_activations_and_types(act, out, bias, residual):
    assert pair_runs(1667, 1544, 160, "nvfp4")
    T.check_gemm(1667, 1544, 160, "nvfp4", out, bias=bias, act=act, preact=True, residual=residual)


@pytest.mark.parametrize("opts", [dict(), dict(bias=F32), dict(act="relu"), dict(preact=True), dict(p=0.5),
                                  dict(residual=F32), dict(p=0.5, residual=BF)], ids=lambda o: "+".join(o) or "none")
@pytest.mark.parametrize("out", [BF, F32], ids=["bf16", "f32"])
def test_pair_epilogue_single_steps(opts, out):
    assert pair_runs(1300, 2056, 320, "mxfp4")
    T.check_gemm(1300, 2056, 320, "mxfp4", out, **opts)


@pytest.mark.parametrize("fmt", list(FMT))
def test_pair_epilogue_without_steps_equals_the_gemm(fmt):
    """No step: the sums of q.gemm, whose kernel is the same but for its last lines."""
    M, N, K = 1667, 1544, 2080
    assert pair_runs(M, N, K, fmt)
    A, B = R.random_operand(M, K, FMT[fmt], 3), R.random_operand(N, K, FMT[fmt], 4)
    for dt in (F32, BF):
        y, z = q.gemm_epilogue(A, B, M, N, K, FMT[fmt], out_dtype=dt)
        assert z is None and torch.equal(y, q.gemm(A, B, M, N, K, FMT[fmt], out_dtype=dt))


@pytest.mark.parametrize("N", [1544, 1600])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_pair_epilogue_residual_in_place(N, dt):
    M, K = 1667, 512
    assert pair_runs(M, N, K, "nvfp4")
    A, B = R.random_operand(M, K, q.NVFP4, 1), R.random_operand(N, K, q.NVFP4, 2)
    r = T.normal((M, N), 3, 100.0, dt)
    kw = dict(bias=T.normal((N,), 4, 100.0), act=q.ACT_SILU, dropout_p=0.2, seed=9)
    want, _ = q.gemm_epilogue(A, B, M, N, K, q.NVFP4, residual=r, out_dtype=dt, **kw)
    got, _ = q.gemm_epilogue(A, B, M, N, K, q.NVFP4, residual=r, out=r, **kw)
    assert got.data_ptr() == r.data_ptr() and torch.equal(got, want)


def test_pair_epilogue_nan_scale_stays_in_its_row():
    M, N, K = 1667, 1544, 320
    assert pair_runs(M, N, K, "mxfp4")
    A, B = R.random_operand(M, K, q.MXFP4, 1), R.random_operand(N, K, q.MXFP4, 2)
    A["scales"][1500, 3] = 255
    for act in T.ACT.values():
        y, _ = q.gemm_epilogue(A, B, M, N, K, q.MXFP4, act=act)
        assert torch.isnan(y).any(1).nonzero().tolist() == [[1500]] and bool(torch.isnan(y[1500]).all())


# ------------------------------------------------------------------ the few-row kernel's column epilogue
# whole k-tiles (128 bytes of a row) and K not split over a cluster: one to three k-tiles, or too many column tiles;
# more than 512 columns, no dropout
@pytest.mark.parametrize("M", [1, 5, 30, 33, 100, 128])
@pytest.mark.parametrize("fmt,N,K", [("nvfp4", 11016, 256), ("nvfp4", 1000, 256), ("mxfp4", 1000, 512),
                                     ("mxfp4", 11016, 1024), ("mxfp8", 1000, 128), ("mxfp8", 11016, 384)])
def test_few_rows_column_epilogue(M, fmt, N, K):
    assert not pair_runs(M, N, K, fmt)
    T.check_gemm(M, N, K, fmt, BF, bias=BF, act="gelu", preact=True, residual=BF)
    T.check_gemm(M, N - 4, K, fmt, F32, bias=F32, act="silu", residual=F32)
    T.check_gemm(M, N, K, fmt, F32, act="gelu_tanh", preact=True, residual=BF)
    T.check_gemm(M, N, K, fmt, BF, bias=F32)


@pytest.mark.parametrize("M,N", [(200, 8200), (515, 2056)])
@pytest.mark.parametrize("fmt", list(FMT))
def test_column_epilogue_of_several_row_tiles(M, N, fmt):
    assert not pair_runs(M, N, 256, fmt)
    T.check_gemm(M, N, 256, fmt, BF, bias=F32, act="relu", preact=True, residual=F32)


@pytest.mark.parametrize("M", [3, 100])
def test_column_epilogue_residual_in_place(M):
    N, K = 11016, 1024
    A, B = R.random_operand(M, K, q.NVFP4, 1), R.random_operand(N, K, q.NVFP4, 2)
    for dt in (BF, F32):
        r = T.normal((M, N), 3, 100.0, dt)
        want, _ = q.gemm_epilogue(A, B, M, N, K, q.NVFP4, act=q.ACT_GELU, residual=r, out_dtype=dt)
        got, _ = q.gemm_epilogue(A, B, M, N, K, q.NVFP4, act=q.ACT_GELU, residual=r, out=r)
        assert got.data_ptr() == r.data_ptr() and torch.equal(got, want)


# ------------------------------------------------------------------ layer norm of many rows
# more than 296 rows: several rows a group at once, the last group incomplete
@pytest.mark.parametrize("M,D", [(301, 256), (303, 512), (302, 1024), (303, 2048), (305, 4096), (309, 8192), (310, 16384),
                                 (315, 32768), (301, 255), (303, 1001), (305, 2047), (307, 4095)])
@pytest.mark.parametrize("dt,wdt", [(BF, F32), (F32, BF)], ids=["bf16", "f32"])
def test_layernorm_forward_of_many_rows(M, D, dt, wdt):
    T.check_layernorm(M, D, dt, wdt)


# odd widths in memory-aligned vectors: rows past the first of a group, groups that end early
@pytest.mark.parametrize("M,D", [(35, 4099), (64, 4101), (70, 5003), (37, 8185), (41, 8195), (70, 16379), (330, 4098),
                                 (331, 6150)])
@pytest.mark.parametrize("dt,wdt", [(BF, F32), (F32, F32), (BF, BF)], ids=["bf16", "f32", "bf16-bf16"])
def test_layernorm_forward_of_odd_long_rows(M, D, dt, wdt):
    T.check_layernorm(M, D, dt, wdt)


@pytest.mark.parametrize("M,D", [(70, 5003), (303, 1001), (305, 4096)])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_layernorm_forward_of_many_rows_in_place(M, D, dt):
    x, g = T.norm_input(M, D, dt), 1 + T.normal((D,), 3, 0.3)
    want, _, _ = q.layernorm_forward(x, g)
    got, _, _ = q.layernorm_forward(x, g, out={"y": x})
    assert torch.equal(got, want)


# ------------------------------------------------------------------ gradients of long rows
@pytest.mark.parametrize("M,D", [(333, 20000), (700, 9001), (150, 16392), (260, 8196), (129, 40001)])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_layernorm_backward_of_long_rows(M, D, dt):
    """Several rows a chunk of the column sums, the last chunk shorter."""
    T.check_layernorm_backward(M, D, dt, F32)


@pytest.mark.parametrize("M,D", [(303, 264), (1201, 520), (601, 1032), (310, 2056), (297, 5120), (299, 12296),
                                 (1203, 255), (900, 1025), (400, 4097), (300, 8191)])
@pytest.mark.parametrize("dt", [BF, F32], ids=["bf16", "f32"])
def test_layernorm_backward_of_many_rows(M, D, dt):
    """Widths between the powers of two, several rows a group."""
    T.check_layernorm_backward(M, D, dt, BF)
