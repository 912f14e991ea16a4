"""Adapters on long rows and wide ranks: the sums behave as binary32 sums do.

An error that a worst-case bound admits may still be far above rounding: one that
always points towards zero grows with the number of additions, while roundings
to nearest partly cancel.  So the rms of the error is held against that of the result.

The limit, in units of u = 2^-24, the relative error of one rounding at most: a
channel slice is a chain of n = ceil(ceil(K / 32) / slices) binary32 additions of
32-channel sums.  A rounding of a partial sum s has an rms of at most u |s| / sqrt(3);
with terms of random sign the mean square of the i-th partial sum is i/n of the
whole, so the chain adds u sqrt(n / 6).  A 32-channel sum is formed by at most four
tensor-core additions of leading parts that may truncate (2 u each, all towards
zero): 8 u.  The parts of two cut operands leave out at most 2^-21 = 8 u of a product.
The sum over the rank does the same once more, in ceil(R / 32) <= 8 steps: sqrt(8 / 6) u,
8 u and 8 u.  Slices are added in at most 16 + 16 additions, u sqrt(32 / 6), and the base
is 0.  Together
  rms(error) <= u (sqrt(n / 6) + 36) rms(result).
"""
import pytest
import torch

import decode_matvec_sq_b200 as sq

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built(cuda_device):
    from decode_matvec_sq_b200 import build
    build.build_all()
    sq.device_check()
    yield
    torch.cuda.empty_cache()


def _slices(M, R):
    """Slices of the channels that a call on M tokens forms at least."""
    if M <= 64:
        return 64
    return 16 // -(-R // 32)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,R,K", [(1300, 128, 4096), (1300, 128, 14336), (1300, 256, 14336), (1300, 256, 65536),
                                   (1300, 33, 14336), (200, 256, 14336), (64, 256, 65536), (5, 64, 14336)])
def test_rms_of_the_error(M, R, K, dtype):
    N, S = 96, 2
    g = torch.Generator(device="cuda").manual_seed(M + R + K)
    A = (torch.randn(S, R, K, generator=g, device="cuda") / K ** 0.5).to(TYPES[dtype])
    B = (0.05 * torch.randn(S, N, R, generator=g, device="cuda")).to(TYPES[dtype])
    x = torch.randn(M, K, generator=g, device="cuda")
    ids = torch.randint(0, S, (M,), generator=g, device="cuda", dtype=torch.int32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = sq.lora_add(sq.LoraBank(A, B, torch.ones(S, device="cuda")), x, ids, status=st)
    assert st.item() == 0
    want = torch.empty(M, N, dtype=torch.float64, device="cuda")
    for a in range(S):
        t = ids == a
        want[t] = (x[t].double() @ A[a].double().t()) @ B[a].double().t()
    err = ((y.double() - want).pow(2).mean().sqrt() / want.pow(2).mean().sqrt()).item()
    n = -(-(-(-K // 32)) // _slices(M, R))
    limit = 2.0 ** -24 * ((n / 6) ** 0.5 + 36)
    assert err <= limit, (err, limit)
