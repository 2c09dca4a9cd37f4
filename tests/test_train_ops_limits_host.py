"""Limits of the grouped products: calls past them are answered on the host,
before anything is launched (no GPU needed)."""
import pytest
import torch

from test_train_ops_host import _dgrad, _gemm, _status, _wgrad, moe  # noqa: F401


@pytest.mark.parametrize("G,N,K", [(1024, 1 << 21, 8),                   # 2^31 weight rows
                                   (1024, (1 << 21) + 8, 16), (1024, 1 << 22, 16), (129, (1 << 24) - 8, 8),
                                   (255, 8421504, 8), (1, 1 << 24, 8)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_weight_rows_that_32_bits_do_not_count(moe, G, N, K, dtype):  # noqa: F811
    """The forward's weight rows are numbered through all the experts, and its
    last tile reaches up to 512 rows behind the last of them."""
    kw = dict(G=G, N=N, K=K, dtype=dtype, out=dtype, n=1 << 50)
    for call in (_gemm, _dgrad, _wgrad):
        assert _status(moe, *call(moe, **kw)) == 2, call.__name__
    for fn in (moe.moe_grouped_workspace_size, moe.moe_grouped_wgrad_workspace_size):
        assert fn(G, N, K, 10, dtype) == 0
        assert fn(1024, (1 << 21) - 8, K, 10, dtype) > 0  # the largest that is open


@pytest.mark.parametrize("n", [1 << 31, (1 << 32) + 4, -(1 << 31) - 1])
def test_sizes_that_32_bits_do_not_hold(moe, n):  # noqa: F811
    """The C interface takes sizes in 32 bits: a larger one is refused, not cut off to its low bits."""
    for make in (lambda: moe.RowCheckpoint(n, 8, torch.bfloat16, device="cuda:0"),
                 lambda: moe.RowCheckpoint(8, n, torch.bfloat16, device="cuda:0"),
                 lambda: moe.ActivationCheckpoint("swiglu", n, 8, torch.bfloat16, device="cuda:0"),
                 lambda: moe.ActivationCheckpoint("gelu_tanh", 8, n, torch.bfloat16, device="cuda:0")):
        with pytest.raises(ValueError, match="32-bit"):
            make()
