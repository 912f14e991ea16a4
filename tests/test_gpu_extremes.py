"""Finite values up to the largest of binary32 in the token-dependent calls: what is
cut into parts stays finite, so the results are those of the formulas."""
import pytest
import torch

import decode_matvec_sq_b200 as sq

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BIG = torch.finfo(torch.float32).max


@pytest.fixture(scope="module", autouse=True)
def built(cuda_device):
    from decode_matvec_sq_b200 import build
    build.build_all()
    sq.device_check()
    yield


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M", [4, 200])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_the_largest_activation_of_an_adapter(M, dtype, sign):
    """One product per sum, by powers of two: v = x 2^-6 or x itself, y = v 2^-10.  The
    parts of x hold all but 2^-21 of it, and so do those of v."""
    K, N, R = 64, 40, 8
    A = torch.zeros(1, R, K, device="cuda")
    A[0, 0, 5], A[0, 1, 6] = 2.0 ** -6, 1.0
    B = torch.zeros(1, N, R, device="cuda")
    B[0, :20, 0], B[0, 20:, 1] = 2.0 ** -10, 2.0 ** -10
    x = torch.zeros(M, K, device="cuda")
    x[:, 5], x[:, 6] = sign * BIG, sign * BIG
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    bank = sq.LoraBank(A.to(TYPES[dtype]), B.to(TYPES[dtype]), torch.ones(1, device="cuda"))
    y = sq.lora_add(bank, x, torch.zeros(M, dtype=torch.int32, device="cuda"), status=st)
    want = torch.full((N,), sign * BIG * 2.0 ** -16, dtype=torch.float64, device="cuda")
    want[20:] *= 2.0 ** 6
    assert st.item() == 0 and ((y.double() - want).abs() <= 2.0 ** -20 * want.abs()).all()


@pytest.mark.parametrize("M", [4, 200])
def test_the_largest_weights_of_an_adapter(M):
    K, N, R = 64, 40, 8
    A = torch.zeros(1, R, K, device="cuda")
    A[0, 0, 5] = BIG
    B = torch.zeros(1, N, R, device="cuda")
    B[0, :, 0] = BIG
    x = torch.zeros(M, K, device="cuda")
    x[:, 5] = 2.0 ** -100
    scale = torch.full((1,), 2.0 ** -60, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = sq.lora_add(sq.LoraBank(A, B, scale), x, torch.zeros(M, dtype=torch.int32, device="cuda"), status=st)
    want = BIG * 2.0 ** -160 * BIG
    assert st.item() == 0 and ((y.double() - want).abs() <= 2.0 ** -20 * want).all()


@pytest.mark.parametrize("n", [6, 100])
@pytest.mark.parametrize("n_out", [1, 40])
def test_the_largest_outlier_activation(n, n_out):
    """Few and many tokens per expert: the outlier channels' products of finite values."""
    N, K = 150, 400
    g = torch.Generator(device="cuda").manual_seed(n + n_out)
    W = 0.02 * torch.randn(N, K, generator=g, device="cuda")
    experts = sq.alloc_experts(1, N, K)
    sq.decompose_pack(W, out=experts.expert(0))
    idx = torch.arange(3, 3 + n_out, dtype=torch.int32, device="cuda")
    x = torch.randn(n, K, generator=g, device="cuda")
    x[1, 3], x[2, 3] = BIG, -BIG
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    q = sq.quantize_act(x, idx, status=st)
    y = sq.grouped_linear(experts, *q, idx, torch.tensor([0, n], dtype=torch.int32, device="cuda"), status=st)
    ref = sq.linear(experts.expert(0), *[v[:4].clone() for v in q], idx, status=st)
    assert st.item() == 0 and torch.isfinite(ref).all()
    # The layer's weight is a sum +-alpha_r + s q of binary32 terms.  s q lies within half a
    # step of W -+ alpha_r, so both terms are at most |W| + 2 alpha_r, and where they cancel
    # (|W| far below alpha_r) a rounding of either, 2^-24 of it, is far above 2e-5 |W|: the
    # two kernels may differ by 2^-22 (|W| + 2 alpha_r) |x|.
    ax, alpha = x[:4].double().abs(), experts.expert(0).alpha().double()
    bound = 2e-5 * (ax @ W.double().abs().t()) + 2.0 ** -22 * (ax @ (W.double().abs() + 2 * alpha[:, None]).t())
    assert ((y[:4].double() - ref.double()).abs() <= bound).all()
