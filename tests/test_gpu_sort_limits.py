"""The sorts at their largest sizes, where one CTA's chunk is full and there are more
chunks than the usual 128, against a stable sort."""
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
    torch.cuda.empty_cache()


def _check(got, ids, S):
    n = ids.numel()
    flat = ids.reshape(-1).long()
    live = int((flat >= 0).sum())
    offsets = torch.bincount(flat[flat >= 0], minlength=S).cumsum(0)
    assert got.offsets[0].item() == 0 and torch.equal(got.offsets[1:].long(), offsets)
    by = torch.sort(torch.where(flat < 0, S, flat), stable=True).indices[:live]
    assert torch.equal(got.order[:live].long(), by) and (got.order[live:] == -1).all()
    place = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    place[by] = torch.arange(live, device="cuda")
    assert torch.equal(got.place.reshape(-1).long(), place)


@pytest.mark.parametrize("n,S", [(524288, 1024), (524289, 1024), (1 << 24, 1024), ((1 << 24) - 5, 3)])
def test_segment_of_the_most_entries(n, S):
    g = torch.Generator(device="cuda").manual_seed(n)
    ids = torch.randint(-1, S, (n,), generator=g, device="cuda", dtype=torch.int32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = sq.segment(ids, S, status=st)
    assert st.item() == 0
    _check(got, ids, S)


@pytest.mark.parametrize("T,E,k", [(1 << 24, 4, 1), (541200, 40, 31), (524288, 64, 32)])
def test_route_of_the_most_entries(T, E, k):
    g = torch.Generator(device="cuda").manual_seed(T)
    logits = torch.randn(T, E, generator=g, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = sq.route(logits, k, status=st)
    assert st.item() == 0
    best = torch.topk(logits, k, dim=1)
    assert torch.equal(torch.gather(logits, 1, got.ids.long()), best.values)  # (equal logits may take turns)
    _check(got, got.ids, E)


def test_one_workspace_for_the_longest_batch():
    E, k, longest = 128, 8, 5001
    ws = torch.empty(sq.lib().sq_route_workspace_bytes(longest, E, k), dtype=torch.uint8, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    logits = torch.randn(longest, E, generator=g, device="cuda")
    for T in (longest, 4097, 4096, 1017, 300, 5):
        got = sq.route(logits[:T], k, workspace=ws)
        _check(got, got.ids, E)
