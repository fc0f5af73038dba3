"""The linear layer at the largest number of rows: more 64×64 tiles than one
launch takes.  Integers: every sum is exact."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16 = torch.bfloat16
M, N, K, PIECE = 1 << 30, 8, 8, 1 << 26


def test_forward_and_dx_of_2_to_the_30_rows(hg):
    """8 columns of 16 bits, 17 GB a matrix."""
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GiB of free GPU memory")
    g = torch.Generator(device=DEV).manual_seed(6)
    X, Y = torch.empty(M, K, dtype=BF16, device=DEV), torch.empty(M, N, dtype=BF16, device=DEV)
    for i in range(0, M, PIECE):
        X[i:i + PIECE] = torch.randint(-2, 3, (PIECE, K), generator=g, device=DEV, dtype=torch.int8)
    W = torch.randint(-2, 3, (N, K), generator=g, device=DEV).to(BF16)
    for w, call in ((W.t(), lambda: hg.linear(X, W, Y)), (W, lambda: hg.linear_grad(X, W, None, dX=Y))):
        Y.fill_(float("nan"))
        call()
        for i in range(0, M, PIECE):
            want = torch.mm(X[i:i + PIECE].float(), w.float().contiguous())     # at most 32: exact in bf16
            assert torch.equal(Y[i:i + PIECE].float(), want), i
