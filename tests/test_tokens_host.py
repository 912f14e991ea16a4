"""Host-side checks of the calls whose weight depends on the token: refusals
before any device work.  No GPU."""
import ctypes

import pytest

import decode_matvec_sq_b200 as sq


@pytest.fixture(scope="module")
def L():
    import torch  # noqa: F401  (loads the CUDA runtime the library links against)
    from decode_matvec_sq_b200 import build
    build.build_libsq()
    return sq.lib()


P = ctypes.c_void_p(1 << 41)
BAD = ctypes.c_void_p((1 << 41) + 4)


def test_route_refusals(L):
    def call(logits=P, T=16, E=64, k=4, gate=0, ids=P, gates=P, offsets=P, order=P, place=P, ws=None, n=0, flags=0):
        return L.sq_route(logits, T, E, k, gate, ids, gates, offsets, order, place, ws, n, None, flags, None)
    for name in ("logits", "ids", "gates", "offsets", "order", "place"):
        assert call(**{name: None}) == 1
        assert call(**{name: BAD}) == 3
    for kw in (dict(T=0), dict(E=0), dict(E=1025), dict(k=0), dict(k=33), dict(E=3), dict(T=1 << 23)):
        assert call(**kw) == 2, kw
    assert call(gate=2) == 1 and call(flags=2) == 1
    # more tokens than one CTA takes: a workspace is needed
    need = L.sq_route_workspace_bytes(5000, 64, 4)
    assert L.sq_route_workspace_bytes(16, 64, 4) == 0 and need > 0 and need % (64 * 4) == 0
    assert call(T=5000) == 8 and call(T=5000, ws=P, n=need - 1) == 8 and call(T=5000, ws=BAD, n=need) == 3


def test_segment_refusals(L):
    def call(ids=P, n=100, S=8, offsets=P, order=P, place=P, ws=None, wn=0, flags=0):
        return L.sq_segment(ids, n, S, offsets, order, place, ws, wn, None, flags, None)
    for name in ("ids", "offsets", "order", "place"):
        assert call(**{name: None}) == 1
        assert call(**{name: BAD}) == 3
    for kw in (dict(n=0), dict(n=(1 << 24) + 1), dict(S=0), dict(S=1025)):
        assert call(**kw) == 2, kw
    assert call(flags=2) == 1
    need = L.sq_segment_workspace_bytes(5000, 8)
    assert need > 0 and call(n=5000) == 8 and call(n=5000, ws=P, wn=need - 1) == 8


def test_combine_refusals(L):
    def call(z=P, rows=8, gates=P, place=P, T=4, k=2, N=64, base=None, out=P, flags=0):
        return L.sq_combine(z, rows, gates, place, T, k, N, base, out, None, flags, None)
    for name in ("z", "gates", "place", "out"):
        assert call(**{name: None}) == 1
        assert call(**{name: BAD}) == 3
    assert call(base=BAD) == 3
    for kw in (dict(rows=0), dict(T=0), dict(k=0), dict(k=33), dict(N=0), dict(T=1 << 24)):
        assert call(**kw) == 2, kw
    assert call(flags=2) == 1


def test_binding_refuses_cpu_tensors_and_wrong_types(L):
    import torch
    for call in (lambda: sq.route(torch.zeros(4, 8), 2), lambda: sq.route(torch.zeros(4, 8), 2, gate="x"),
                 lambda: sq.segment(torch.zeros(4), 2), lambda: sq.segment(torch.zeros(4, dtype=torch.int32), 2),
                 lambda: sq.combine(torch.zeros(4, 8), torch.zeros(2, 2), torch.zeros(2, 2, dtype=torch.int32))):
        with pytest.raises(sq.SQError):
            call()
