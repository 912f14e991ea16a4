"""The token-dependent calls where element offsets pass 32 bits, and at the longest
rows: compared on the last rows, where a wrapped offset would show."""
import numpy as np
import pytest
import torch

import decode_matvec_sq_b200 as sq
import oracle

pytestmark = pytest.mark.gpu

TOL = 1e-5


@pytest.fixture(scope="module", autouse=True)
def built(cuda_device):
    from decode_matvec_sq_b200 import build
    build.build_all()
    sq.device_check()
    yield
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n", [5, 960])
def test_the_last_expert_of_a_stack_past_32_bits(n):
    E, N, K = 40, 4096, 14336
    assert E * N * K > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(n)
    experts = sq.alloc_experts(E, N, K)
    W = 0.02 * torch.randn(N, K, generator=g, device="cuda")
    sq.decompose_pack(W, out=experts.expert(E - 1))
    x = torch.randn(n, K, generator=g, device="cuda")
    idx = torch.tensor([0, 777, K - 1], dtype=torch.int32, device="cuda")
    q = sq.quantize_act(x, idx)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[E] = n
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = sq.grouped_linear(experts, *q, idx, off, status=st)
    at = slice(max(0, n - 16) // 4 * 4, n)
    ref = sq.linear(experts.expert(E - 1), *[v[at].clone() for v in q], idx)
    bound = x[at].double().abs() @ W.double().abs().t()
    assert st.item() == 0 and ((y[at] - ref).abs() <= 2 * TOL * bound).all()


def test_rows_of_y_past_32_bits():
    N, K, n = 4096, 128, 600_000
    assert n * N > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(1)
    experts = sq.alloc_experts(1, N, K)
    W = 0.02 * torch.randn(N, K, generator=g, device="cuda")
    sq.decompose_pack(W, out=experts.expert(0))
    x = torch.randn(n, K, generator=g, device="cuda")
    q = sq.quantize_act(x, None)
    off = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    z = sq.grouped_linear(experts, *q, None, off, status=st)
    at = slice(n - 16, n)
    ref = sq.linear(experts.expert(0), *[v[at].clone() for v in q], None)
    bound = x[at].double().abs() @ W.double().abs().t()
    assert st.item() == 0 and ((z[at] - ref).abs() <= 2 * TOL * bound).all()
    # and back to tokens: the last token takes the last row and the first
    place = torch.tensor([[n - 1, 0], [n - 2, -1]], dtype=torch.int32, device="cuda")
    out = sq.combine(z, torch.ones(2, 2, device="cuda"), place, status=st)
    assert st.item() == 0 and torch.equal(out[0], z[n - 1] + z[0]) and torch.equal(out[1], z[n - 2])


def test_adapter_rows_past_32_bits():
    M, N, K, R = 600_000, 4096, 32, 4
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").float()  # every sum is exact
    bank = sq.LoraBank(rnd(2, R, K), rnd(2, N, R), torch.ones(2, device="cuda"))
    x = rnd(M, K)
    ids = torch.randint(-1, 2, (M,), generator=g, device="cuda", dtype=torch.int32)
    y = torch.ones(M, N, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    sq.lora_add(bank, x, ids, base=y, y=y, status=st)
    at = slice(M - 64, M)
    a = ids[at].clamp(min=0).long()
    v = (bank.A[a] * x[at, None, :]).sum(2)
    want = 1.0 + torch.where(ids[at, None] >= 0, (bank.B[a] * v[:, None, :]).sum(2), 0.0)
    assert st.item() == 0 and torch.equal(y[at], want)


@pytest.mark.parametrize("n", [3, 30])
def test_the_longest_rows(n):
    """131072 channels: 1024 groups, a binary32 chain of as many terms."""
    N, K = 20, 131072
    rng = np.random.default_rng(n)
    W, x = rng.laplace(0, 0.02, (N, K)).astype(np.float32), rng.standard_normal((n, K)).astype(np.float32)
    idx = np.array([5, 70000, K - 1], np.int32)
    x[:, idx] *= 30.0
    experts = sq.alloc_experts(1, N, K)
    sq.decompose_pack(torch.from_numpy(W).cuda(), out=experts.expert(0))
    idxd = torch.from_numpy(idx).cuda()
    q = sq.quantize_act(torch.from_numpy(x).cuda(), idxd)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = sq.grouped_linear(experts, *q, idxd, torch.tensor([0, n], dtype=torch.int32, device="cuda"), status=st)
    ref = oracle.linear(oracle.decompose(W), *oracle.quantize_act(x, idx), idx)
    err = np.abs(y.cpu().numpy().astype(np.float64) - ref)
    assert st.item() == 0 and (err <= (K / 128 + 16) * 2.0 ** -24 * oracle.abs_dot(W, x)).all()
