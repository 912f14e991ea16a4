"""The grouped layer on stacks of many experts, with an asymmetric residual at many tokens,
and with fewer tiles than the device has SMs over long rows; tolerances as in
test_gpu_grouped.py (1e-5 of the sum of magnitudes, 112 groups at most)."""
import pytest
import torch

import decode_matvec_sq_b200 as sq
from test_gpu_grouped import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built(cuda_device):
    from decode_matvec_sq_b200 import build
    build.build_all()
    sq.device_check()
    yield


@pytest.mark.parametrize("n_out", [0, 20])
def test_few_tiles_over_long_rows(n_out):
    c = Case(4, 130, 14336, [40, 0, 150, 30], n_out=n_out, spare=2)
    c.check(c.run())


@pytest.mark.parametrize("layout", [sq.SQ_LAYOUT_TILES, sq.SQ_LAYOUT_TILES_ASYM])
@pytest.mark.parametrize("n_out", [143, 300])
def test_more_outlier_channels_than_the_many_token_kernel_takes(n_out, layout):
    c = Case(2, 40, 2048, [70, 33], layout=layout, n_out=n_out)
    c.check(c.run())


@pytest.mark.parametrize("E,hot", [(128, 200), (256, 40)])
def test_many_experts_one_of_them_hot(E, hot):
    """Most experts without a token; fewer than 24 places an expert on average."""
    counts = [0] * E
    counts[3], counts[E // 2], counts[E - 1] = 1, hot, 2
    c = Case(E, 24, 300, counts, n_out=3, spare=1)
    c.check(c.run())


def test_asymmetric_residual_with_hundreds_of_tokens():
    c = Case(3, 100, 700, [300, 0, 120], layout=sq.SQ_LAYOUT_TILES_ASYM, P=60, n_out=9)
    assert torch.equal(c.run(), c.run())
    c.check(c.run())
