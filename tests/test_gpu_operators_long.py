"""Column sums over very many rows: no running sum takes more than 2048 terms."""
import pytest
import torch

import bit_fwht_hadamard_b200 as q

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
# a running sum of 2048 terms, the groups of a block (8 at most), a lane's partial rows (512 at most here), a tree of
# five levels; with terms of one sign a chain of 16000 is off by 3400 u
TERMS = (2048 + 8 + 512 + 8) * U
C = 0.37


@pytest.mark.parametrize("M,N", [(1 << 26, 3), (131072, 75776)])
def test_bias_gradient_of_many_rows(M, N):
    dy = torch.full((M, N), C, device="cuda")
    _, db = q.epilogue_backward(dy, out={"dZ": dy})
    want = M * float(torch.tensor(C))
    assert float((db.double() - want).abs().max()) <= TERMS * want


# three odd columns, the ring of bulk copies, rows longer than any group
@pytest.mark.parametrize("M,D", [(1 << 26, 3), (9_800_000, 520), (80000, 65536)])
def test_norm_gradients_of_many_rows(M, D):
    dy = torch.full((M, D), C, device="cuda")
    row = torch.linspace(0.5, 1.5, D, device="cuda")
    x = row.expand(M, D).contiguous()
    zero, one = torch.zeros(M, device="cuda"), torch.ones(M, device="cuda")
    _, dg, db = q.layernorm_backward(dy, x, None, zero, one, want_dx=False)
    want = M * float(torch.tensor(C))
    assert float((db.double() - want).abs().max()) <= TERMS * want
    assert float(((dg.double() - want * row.double()) / (want * row.double())).abs().max()) <= TERMS + 2 * U
    assert q.qfp4_last_device_error() == 0
