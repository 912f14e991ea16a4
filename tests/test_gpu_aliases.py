"""Results written over an input, where the calls allow it, and refused where not."""
import pytest
import torch

import decode_matvec_sq_b200 as sq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built(cuda_device):
    from decode_matvec_sq_b200 import build
    build.build_all()
    sq.device_check()
    yield


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("with_base", ["none", "x", "other"])
@pytest.mark.parametrize("M,N,col", [(1, 256, 0), (1, 100, 7), (5, 256, 0), (64, 200, 0), (33, 200, 56), (65, 256, 0),
                                     (400, 256, 0), (700, 100, 3)])
def test_adapters_over_their_own_activations(M, N, col, with_base, dtype):
    """y is x or columns of it: rows are read before they are written, other columns stay."""
    K, S, R = 256, 3, 16
    g = torch.Generator(device="cuda").manual_seed(M)
    bank = sq.LoraBank(torch.randn(S, R, K, generator=g, device="cuda").to(dtype),
                       torch.randn(S, N, R, generator=g, device="cuda").to(dtype), torch.ones(S, device="cuda"))
    x = torch.randn(M, K, generator=g, device="cuda")
    ids = torch.randint(-1, S, (M,), generator=g, device="cuda", dtype=torch.int32)
    base = {"none": None, "x": x[:, col:col + N].clone(), "other": torch.randn(M, N, generator=g, device="cuda")}[with_base]
    want = sq.lora_add(bank, x, ids, base=base)
    z = x.clone()
    part = z[:, col:col + N]
    sq.lora_add(bank, z, ids, base=part if with_base == "x" else base, y=part)
    assert torch.equal(part, want)
    part.copy_(x[:, col:col + N])
    assert torch.equal(z, x)


def test_results_over_other_inputs_are_refused():
    z = torch.randn(6, 32, device="cuda")
    place = torch.tensor([[0], [1]], dtype=torch.int32, device="cuda")
    gates = torch.ones(2, 1, device="cuda")
    with pytest.raises(sq.SQError):
        sq.combine(z, gates, place, out=z[:2])
    wide = torch.zeros(3, 32, device="cuda")
    with pytest.raises(sq.SQError):
        sq.combine(z, gates, place, base=wide[:2], out=wide[1:])
    bank = sq.LoraBank(torch.zeros(1, 8, 32, device="cuda"), torch.zeros(1, 16, 8, device="cuda"), torch.ones(1, device="cuda"))
    qkv, ids = torch.zeros(6, 48, device="cuda"), torch.zeros(6, dtype=torch.int32, device="cuda")
    with pytest.raises(sq.SQError):
        sq.lora_add(bank, z, ids, base=qkv[:, 8:24], y=qkv[:, 16:32])
    out = sq.lora_add(bank, z, ids, base=qkv[:, :16], y=qkv[:, 16:32])
    assert out.data_ptr() == qkv.data_ptr() + 64
