"""The token-dependent calls on a stream other than the current one: results and
scratch come from that stream's memory, and the numbers are those of the current
stream."""
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


def _calls():
    g = torch.Generator(device="cuda").manual_seed(1)
    T, E, k, N, K, S = 300, 4, 2, 200, 256, 5
    logits = torch.randn(T, E, generator=g, device="cuda")
    r = sq.route(logits, k)
    experts = sq.alloc_experts(E, N, K)
    for e in range(E):
        sq.decompose_pack(torch.randn(N, K, generator=g, device="cuda"), out=experts.expert(e))
    idx = torch.tensor([3, 9], dtype=torch.int32, device="cuda")
    q = sq.quantize_act(torch.randn(T, K, generator=g, device="cuda"), idx)
    z = torch.randn(T * k, N, generator=g, device="cuda")
    bank = sq.LoraBank(torch.randn(S, 8, K, generator=g, device="cuda"), torch.randn(S, N, 8, generator=g, device="cuda"),
                       torch.ones(S, device="cuda"))
    x = torch.randn(T, K, generator=g, device="cuda")
    ids = torch.randint(-1, S, (T,), generator=g, device="cuda", dtype=torch.int32)
    many = torch.randint(-1, S, (5000,), generator=g, device="cuda", dtype=torch.int32)
    torch.cuda.synchronize()
    return {
        "route": lambda **kw: sq.route(logits, k, **kw).gates,
        "segment": lambda **kw: sq.segment(many, S, **kw).order,
        "grouped_linear": lambda **kw: sq.grouped_linear(experts, *q, idx, r.offsets, order=r.order, div=k, **kw),
        "combine": lambda **kw: sq.combine(z, r.gates, r.place, **kw),
        "lora_add": lambda **kw: sq.lora_add(bank, x, ids, **kw),
    }


@pytest.mark.parametrize("name", ["route", "segment", "grouped_linear", "combine", "lora_add"])
def test_results_come_from_the_named_streams_memory(name):
    call = _calls()[name]
    ref = call()
    torch.cuda.synchronize()
    freed = [torch.empty_like(ref) for _ in range(64)]  # blocks the current stream would be given again
    at = {t.untyped_storage().data_ptr() for t in freed}
    base = {t.data_ptr() // (2 << 20) for t in freed}
    del freed
    s = torch.cuda.Stream()
    y = call(stream=s)
    s.synchronize()
    assert torch.equal(y, ref)
    assert y.untyped_storage().data_ptr() not in at and y.data_ptr() // (2 << 20) not in base


@pytest.mark.parametrize("name", ["route", "segment", "grouped_linear", "combine", "lora_add"])
def test_scratch_is_not_handed_out_while_the_call_runs(name):
    """Many calls on two other streams, each with scratch of its own, against the
    same on the current stream."""
    call = _calls()[name]
    ref = call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ys = [call(stream=streams[i % 2]) for i in range(20)]
    torch.cuda.synchronize()
    for y in ys:
        assert torch.equal(y, ref)


def test_weights_that_are_not_on_the_current_device_are_refused():
    experts = sq.alloc_experts(2, 32, 128)
    experts.keep = (experts.keep[0].cpu(),)
    q = sq.quantize_act(torch.randn(4, 128, device="cuda"), None)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    with pytest.raises(sq.SQError, match="experts are not on the current device"):
        sq.grouped_linear(experts, *q, None, off)
    bank = sq.LoraBank(torch.zeros(1, 8, 128, device="cuda"), torch.zeros(1, 16, 8, device="cuda"),
                       torch.ones(1, device="cuda"))
    bank.A = bank.A.cpu()
    with pytest.raises(sq.SQError, match="adapters are not on the current device"):
        sq.lora_add(bank, torch.zeros(4, 128, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda"))
