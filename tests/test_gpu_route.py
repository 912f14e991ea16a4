"""The router, the sort of entries into segments and the weighted sum of the
experts' rows, against plain numpy in 64 bits.

ids, offsets, order and place are whole numbers and must be equal.  Gates: a
binary32 exp within 2 ulp, a sum of at most E <= 1024 terms (each addition half
an ulp) and one division: relative error below (2 + 2 + log2-depth sums of at
most 32 + 5 additions + 1) * 2^-24 < 64 * 2^-24.  The sum of rows: k <= 32 fused
multiply-adds and one addition, so within (k + 1) * 2^-24 of the sum of
magnitudes.
"""
import numpy as np
import pytest
import torch

import decode_matvec_sq_b200 as sq

pytestmark = pytest.mark.gpu

GATE_TOL = 64 * 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def built(cuda_device):
    from decode_matvec_sq_b200 import build
    build.build_all()
    sq.device_check()
    yield


def _sorted(ids, S):
    """offsets, order, place of ids (flat, -1 = none)."""
    n = ids.size
    live = np.flatnonzero(ids >= 0)
    by = live[np.argsort(ids[live], kind="stable")]
    order = np.full(n, -1, np.int64)
    order[:by.size] = by
    place = np.full(n, -1, np.int64)
    place[by] = np.arange(by.size)
    offsets = np.concatenate([[0], np.cumsum(np.bincount(ids[live], minlength=S))])
    return offsets, order, place


def _routed(logits, k, gate):
    """ids and gates: the largest first, ties to the lower expert; -inf and NaN masked."""
    T, E = logits.shape
    l = logits.astype(np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    ids = np.full((T, k), -1, np.int64)
    gates = np.zeros((T, k))
    for t in range(T):
        best = [e for e in np.argsort(-l[t], kind="stable")[:k] if l[t, e] > -np.inf]
        if not best:
            continue
        ids[t, :len(best)] = best
        with np.errstate(invalid="ignore"):
            over = np.where(l[t] == l[t, best[0]], 1.0, np.exp(l[t] - l[t, best[0]]))
        over[l[t] == -np.inf] = 0.0
        gates[t, :len(best)] = over[best] / (over[best].sum() if gate == "topk" else over.sum())
    return ids, gates


def _check_sort(got, ids, S):
    offsets, order, place = _sorted(ids.reshape(-1), S)
    np.testing.assert_array_equal(got.offsets.cpu().numpy(), offsets)
    np.testing.assert_array_equal(got.order.cpu().numpy(), order)
    np.testing.assert_array_equal(got.place.cpu().numpy().reshape(-1), place)


@pytest.mark.parametrize("gate", ["topk", "all"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (16, 64, 4), (33, 33, 7), (256, 128, 16), (257, 100, 8),
                                   (300, 1024, 32), (5, 1000, 3), (4099, 128, 2), (20000, 17, 5)])
def test_route(T, E, k, gate):
    rng = np.random.default_rng(T + E + k)
    logits = (np.round(rng.standard_normal((T, E)) * 6) / 4).astype(np.float32)  # many ties
    logits[rng.random((T, E)) < 0.1] = -np.inf
    logits[rng.random((T, E)) < 0.05] = np.float32(np.finfo(np.float32).min)
    logits[rng.random((T, E)) < 0.05] *= 0.0  # zeros of both signs tie (and -inf * 0 = NaN)
    logits[0] = -np.inf if T > 1 else logits[0]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = sq.route(torch.from_numpy(logits).cuda(), k, gate=gate, status=st)
    ids, gates = _routed(logits, k, gate)
    assert st.item() == (6 if np.isnan(logits).any() else 0)
    np.testing.assert_array_equal(r.ids.cpu().numpy(), ids)
    np.testing.assert_allclose(r.gates.cpu().numpy(), gates, rtol=GATE_TOL, atol=1e-37)
    _check_sort(r, ids, E)


def test_route_infinite_logits_take_the_limit():
    logits = np.zeros((2, 5), np.float32)
    logits[0, [1, 3]] = np.inf
    logits[1, 2] = np.inf
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = sq.route(torch.from_numpy(logits).cuda(), 2, status=st)
    assert st.item() == 6
    assert r.ids.cpu().tolist() == [[1, 3], [2, 0]]
    assert r.gates.cpu().tolist() == [[0.5, 0.5], [1.0, 0.0]]


@pytest.mark.parametrize("n,S", [(1, 1), (31, 3), (1000, 1024), (4096, 7), (4097, 7), (100003, 33), (300000, 1024)])
@pytest.mark.parametrize("kind", ["mixed", "one", "none"])
def test_segment(n, S, kind):
    rng = np.random.default_rng(n + S)
    ids = {"mixed": rng.integers(-1, S, n), "one": np.full(n, S - 1), "none": np.full(n, -1)}[kind].astype(np.int32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = sq.segment(torch.from_numpy(ids).cuda(), S, status=st)
    assert st.item() == 0
    _check_sort(got, ids, S)


@pytest.mark.parametrize("n", [100, 9000])
def test_segment_reports_ids_out_of_range(n):
    rng = np.random.default_rng(n)
    ids = rng.integers(0, 8, n).astype(np.int32)
    ids[[3, 50, n - 1]] = [8, -2, 2 ** 30]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = sq.segment(torch.from_numpy(ids).cuda(), 8, status=st)
    assert st.item() == 1
    ids[[3, 50, n - 1]] = -1
    _check_sort(got, ids, 8)


@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (1, 2, 4096), (16, 2, 4096), (7, 32, 1028), (33, 5, 1001), (500, 4, 2050)])
@pytest.mark.parametrize("base", ["none", "other", "out"])
def test_combine(T, k, N, base):
    rng = np.random.default_rng(T + k + N)
    z = rng.standard_normal((T * k, N)).astype(np.float32)
    place = rng.permutation(T * k).reshape(T, k).astype(np.int32)
    place[rng.random((T, k)) < 0.2] = -1
    gates = rng.random((T, k)).astype(np.float32)
    gates[place < 0] = np.nan  # never used
    unused = np.setdiff1d(np.arange(T * k), place[place >= 0])
    z[unused] = np.nan
    b = rng.standard_normal((T, N)).astype(np.float32) if base != "none" else np.zeros((T, N), np.float32)
    g = np.where(place >= 0, gates, 0).astype(np.float64)
    rows = np.where((place >= 0)[..., None], z[np.maximum(place, 0)], 0).astype(np.float64)
    want = b + (g[..., None] * rows).sum(1)
    mag = np.abs(b) + (g[..., None] * np.abs(rows)).sum(1)
    bd = torch.from_numpy(b).cuda()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = sq.combine(torch.from_numpy(z).cuda(), torch.from_numpy(gates).cuda(), torch.from_numpy(place).cuda(),
                     base=None if base == "none" else bd, out=bd if base == "out" else None, status=st)
    assert st.item() == 0
    assert (np.abs(out.cpu().numpy() - want) <= (k + 1) * 2.0 ** -24 * mag).all()


def test_combine_reports_places_out_of_range():
    z = torch.ones(4, 8, device="cuda")
    place = torch.tensor([[0, 4], [-2, 1]], dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = sq.combine(z, torch.ones(2, 2, device="cuda"), place, status=st)
    assert st.item() == 1
    assert (out == 1).all()


def test_route_and_combine_in_a_graph_and_back_to_back():
    """Captured with programmatic dependent launches and replayed on new
    logits; results equal those of plain calls."""
    T, E, k, N = 64, 32, 4, 512
    gen = torch.Generator(device="cuda").manual_seed(1)
    logits = torch.randn(T, E, device="cuda", generator=gen)
    z = torch.randn(T * k, N, device="cuda", generator=gen)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sq.combine(z, sq.route(logits, k).gates, sq.route(logits, k).place)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            r = sq.route(logits, k, pdl=True)
            out = sq.combine(z, r.gates, r.place, pdl=True)
    for seed in range(3):
        logits.copy_(torch.randn(T, E, device="cuda", generator=gen))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        want = sq.route(logits, k)
        torch.testing.assert_close(r.order, want.order, rtol=0, atol=0)
        torch.testing.assert_close(out, sq.combine(z, want.gates, want.place), rtol=0, atol=0)
