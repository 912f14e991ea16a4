"""A layer of experts whose routes drop entries (masked experts), over memory that
held something else before: rows that no token has must not show anywhere."""
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


def _layer(T, E, k, D, H, masked, layout=sq.SQ_LAYOUT_TILES):
    g = torch.Generator(device="cuda").manual_seed(T + E)
    up, down = sq.alloc_experts(E, H, D, layout=layout), sq.alloc_experts(E, D, H, layout=layout)
    for e in range(E):
        sq.decompose_pack(0.05 * torch.randn(H, D, generator=g, device="cuda"), out=up.expert(e))
        sq.decompose_pack(0.05 * torch.randn(D, H, generator=g, device="cuda"), out=down.expert(e))
    x = torch.randn(T, D, generator=g, device="cuda")
    logits = torch.randn(T, E, generator=g, device="cuda")
    logits[:, masked:] = float("-inf")
    return up, down, x, logits


def _nan_memory(*shapes):
    """Blocks of these shapes, full of NaN, go back to the allocator."""
    blocks = [torch.full(s, float("nan"), device="cuda") for s in shapes for _ in range(3)]
    torch.cuda.synchronize()
    del blocks


@pytest.mark.parametrize("layout", [sq.SQ_LAYOUT_TILES, sq.SQ_LAYOUT_TILES_ASYM])
@pytest.mark.parametrize("T,E,masked", [(7, 4, 1), (3, 40, 1), (200, 4, 1), (333, 4, 0), (5, 4, 0)])
def test_dropped_entries_leave_no_trace(T, E, masked, layout):
    """k = 2 choices, `masked` experts open: at least half of the entries have no place."""
    k, D, H = 2, 256, 384
    up, down, x, logits = _layer(T, E, k, D, H, masked, layout)
    idx = torch.tensor([3, 200], dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = sq.route(logits, k, status=st)
    q1 = sq.quantize_act(x, idx, status=st)
    live = int(r.offsets[E])
    assert live == T * masked
    _nan_memory((T * k, H), (T * k, D))
    h = sq.grouped_linear(up, *q1, idx, r.offsets, order=r.order, div=k, status=st)
    assert (h[live:] == 0).all()
    q2 = sq.quantize_act(torch.nn.functional.silu(h), idx, status=st)
    _nan_memory((T * k, D))
    z = sq.grouped_linear(down, *q2, idx, r.offsets, status=st)
    assert (z[live:] == 0).all()
    out = sq.combine(z, r.gates, r.place, base=x, status=st)
    assert st.item() == 0 and torch.isfinite(out).all()
    if masked == 0:
        assert torch.equal(out, x)


@pytest.mark.parametrize("T", [4, 150])
def test_rows_of_a_tensor_of_ones_own_stay(T):
    up, _, x, logits = _layer(T, 3, 2, 128, 96, 1)
    r = sq.route(logits, 2)
    y = torch.full((2 * T, 96), 7.0, device="cuda")
    sq.grouped_linear(up, *sq.quantize_act(x, None), None, r.offsets, order=r.order, div=2, y=y)
    assert (y[int(r.offsets[3]):] == 7.0).all()
