"""The bias gradient by itself: what it does not read need not be given."""

import pytest
import torch

from transformer_block_gb300 import pb

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    torch.cuda.set_device(0)
    pb.lib()


@pytest.mark.parametrize("m,n", [(1, 8), (32, 77), (33, 264), (2000, 1000)])
@pytest.mark.parametrize("layout", [pb.PB_WEIGHT_IN_OUT, pb.PB_WEIGHT_OUT_IN])
def test_bias_gradient_without_operands(m, n, layout):
    g = torch.Generator(device="cuda").manual_seed(m)
    dy = torch.randn(m, n + -n % 8, generator=g, device="cuda").to(torch.bfloat16)[:, :n]
    dx, dw, db = pb.linear_backward(dy, None, None, layout=layout, need_dx=False, need_dw=False,
                                    bias=True)
    assert dx is None and dw is None
    # each thread adds rows / 512 values or so, then 8 threads and 8 parts: one rounding each
    room = (m / 512 + 80) * 2.0 ** -24 * dy.double().abs().sum(0)
    assert ((db.double() - dy.double().sum(0)).abs() <= room).all()
    again = pb.linear_backward(dy, None, None, layout=layout, need_dx=False, need_dw=False,
                               db=db.clone(), accumulate=True)[2]
    assert torch.equal(again, db + db)
    with pytest.raises(ValueError, match="needs w"):
        pb.linear_backward(dy, dy, None, layout=layout, need_dw=False)
    with pytest.raises(ValueError, match="needs x"):
        pb.linear_backward(dy, None, dy, layout=layout, need_dx=False)
