"""Where the 16-bit operand of a gradient's products ends: dz = dY·act'(z) past
the type's largest value is infinite in the products, as any value rounded to
the type is, and finite in dbias, which sums it unrounded."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("name", ["GELU", "GELU_TANH", "SILU"])
@pytest.mark.parametrize("M,N,K", [(3, 40, 64), (70, 136, 200)])
def test_dz_past_fp16(hg, M, N, K, name):
    """At z = 2 the slopes are 1.085, 1.086 and 1.091: dY = 61 000 is finite and dz above 65 520 is not, dY = 59 000
    stays below (64 600 at most)."""
    t = torch.float16
    Z, dY = torch.full((M, N), 2.0, dtype=t, device=DEV), torch.zeros(M, N, dtype=t, device=DEV)
    dY[1, 3], dY[2, 5] = 61000.0, 59000.0
    W, X = torch.full((N, K), 2.0 ** -4, dtype=t, device=DEV), torch.full((M, K), 2.0 ** -4, dtype=t, device=DEV)
    dX, dW, db = torch.empty_like(X), torch.empty(N, K, device=DEV), torch.empty(N, device=DEV)
    hg.linear_grad(dY, W, X, Z=Z, act=getattr(hg, "ACT_" + name), dX=dX, dW=dW, dbias=db)
    inf = float("inf")
    assert (dX[1] == inf).all() and dX[2].isfinite().all() and (dX[0] == 0).all() and (dX[3:] == 0).all()
    assert (dW[3] == inf).all() and dW[5].isfinite().all() and (dW[:3] == 0).all()
    assert 65520 < float(db[3]) < 67000 and 63000 < float(db[5]) < 65520
    hg.linear_grad(dY.bfloat16(), W.bfloat16(), X.bfloat16(), Z=Z.bfloat16(), act=getattr(hg, "ACT_" + name),
                   dX=dX.bfloat16().zero_(), dW=dW, dbias=db)
    assert dW.isfinite().all()                              # bfloat16 has the range
