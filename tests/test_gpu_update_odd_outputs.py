"""The orthogonalised update into matrices that TMA cannot address, of so many tiles that each warp's buffer holds outputs by
ordinary stores and then the next tile's R by TMA: the same bits as into a matrix that TMA stores."""
import numpy as np
import pytest
import torch

from trend_util import matrix

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("K,N", [(2600, 2700), (3100, 2305)])
def test_odd_outputs_have_the_same_bits(lib, out, K, N):
    G = torch.randn(N, K, generator=torch.Generator(device="cuda").manual_seed(K), device="cuda").T
    want = lib.orthogonalize(G, 2, out_dtype=out)
    assert torch.isfinite(want).all()
    for pad, shift in ((1, 0), (0, 1), (3, 5)):
        place = matrix(np.zeros((K, N)), out, pad, shift)
        around = place._base.isnan()
        for _ in range(8):
            place.zero_()
            assert lib.orthogonalize(G, 2, out=place) is place
            assert torch.equal(place, want)
        assert torch.equal(place._base.isnan(), around)   # padding and surroundings are left alone
