"""The group norm at the largest number of features and groups: feature blocks and groups together pass 2^31."""
import pytest
import torch

pytestmark = pytest.mark.gpu


def test_a_group_per_feature_at_the_largest_size(lib):
    """One site and one feature per group: the mean is the value, nothing deviates, and the gradient is 0."""
    D = 2 ** 31 - 2 ** 16
    X = torch.empty(1, D, dtype=torch.float16, device="cuda").normal_().T
    try:
        Y, mean, rstd = lib.group_norm(X, D, eps=0.25, save=True)
        assert not Y.any() and torch.equal(mean.half(), X) and bool((rstd == 2.0).all())
        dX, _, _ = lib.group_norm_backward(X, D, None, None, X, mean, rstd, need=(True, False, False))
        assert not dX.any()
    finally:
        torch.cuda.synchronize()
        lib.workspace_trim()
        X = Y = mean = rstd = dX = None
        torch.cuda.empty_cache()
