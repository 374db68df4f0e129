"""Values that no C structure of the state-space block's calls can hold are the caller's errors."""
import pytest
import torch

import zero_order_recurrent_b200 as zo

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def library():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from zero_order_recurrent_b200 import build
    build.build()
    zo.load_library()


@pytest.mark.parametrize("eps", [1e39, -1e300, "1e-6", None])
def test_eps_that_is_no_fp32(eps):
    x, w = torch.ones(2, 8, device="cuda"), torch.ones(8, device="cuda")
    with pytest.raises((ValueError, zo.ZOError)):
        zo.zo_block_norm(x, n_out=torch.empty_like(x), w_pre=w, eps=eps)
    with pytest.raises((ValueError, zo.ZOError)):
        zo.zo_block_norm_backward(x, dn=x, dx=torch.empty_like(x), w_pre=w, dw_pre=w.clone(), eps=eps)


def test_more_rows_than_an_int_holds():
    n = 2 ** 31  # (one element of memory)
    x, y = (torch.ones(1, 1, device="cuda").expand(n, 1) for _ in range(2))
    w = torch.ones(1, device="cuda")
    with pytest.raises(ValueError):
        zo.zo_block_norm(x, n_out=y, w_pre=w)
    x3 = torch.ones(1, 1, 1, device="cuda").expand(n, 1, 1)
    with pytest.raises(ValueError):
        zo.zo_conv(x3, w[None], x3)
    with pytest.raises(ValueError):
        zo.zo_conv_backward(x3, w[None], x3, x3, w[None])
    bc = x3[..., None]
    with pytest.raises(ValueError):
        zo.zo_scan(x3, x3, w[None], bc, bc, x3)
