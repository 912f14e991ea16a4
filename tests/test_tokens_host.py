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


def _stack(L, E=4, N=30, K=300, mask=0, layout=1):
    v = sq.SqPackedWeight()
    assert L.sq_packed_view(ctypes.c_void_p(1 << 40), E * sq.round_up(N, 16), K, 128, mask, layout, ctypes.byref(v)) == 0
    return v


@pytest.mark.parametrize("mask", [0, 1])
@pytest.mark.parametrize("layout", [sq.SQ_LAYOUT_TILES, sq.SQ_LAYOUT_TILES_ASYM])
def test_expert_view(L, mask, layout):
    v, e = _stack(L, mask=mask, layout=layout), sq.SqPackedWeight()
    assert L.sq_expert_view(ctypes.byref(v), 4, 30, 3, ctypes.byref(e)) == 0
    assert (e.N, e.K, e.layout, e.res_stride) == (30, 300, layout, 384)
    assert e.res_q - v.res_q == 96 * 384 and e.sign_bits - v.sign_bits == 96 * 12 * 4
    assert e.alpha - v.alpha == 96 * 4 and e.res_scale - v.res_scale == 96 * 3 * 4
    assert (e.mask_bits is None) == (mask == 0)
    if mask:
        assert e.mask_bits - v.mask_bits == 96 * 12 * 4
    if layout == sq.SQ_LAYOUT_TILES_ASYM:
        assert e.res_zero - v.res_zero == 96 * 3 * 4
    for args in ((4, 30, 4), (4, 30, -1)):
        assert L.sq_expert_view(ctypes.byref(v), *args, ctypes.byref(e)) == 1
    for args in ((4, 33, 0), (3, 30, 0), (0, 30, 0), (1025, 30, 0)):
        assert L.sq_expert_view(ctypes.byref(v), *args, ctypes.byref(e)) == 2
    rows, sparse = _stack(L, layout=0), _stack(L, layout=2)
    for w in (rows, sparse):
        assert L.sq_expert_view(ctypes.byref(w), 4, 30, 0, ctypes.byref(e)) == 1


def test_grouped_linear_refusals(L):
    v = _stack(L)

    def call(stack=v, E=4, N=30, xq=P, sx=P, xo=P, idx=P, n_out=2, rows=8, order=P, div=2, off=P, n=16, y=P, ws=P,
             wn=1 << 30, flags=0):
        return L.sq_grouped_linear(None if stack is None else ctypes.byref(stack), E, N, xq, sx, xo, idx, n_out, rows,
                                   order, div, off, n, y, ws, wn, None, flags, None)
    assert call(stack=None) == 1 and call(stack=_stack(L, layout=0)) == 1 and call(stack=_stack(L, layout=2)) == 1
    for name in ("xq", "sx", "xo", "idx", "off", "y"):
        assert call(**{name: None}) == 1, name
        assert call(**{name: BAD}) == 3, name
    assert call(order=BAD) == 3 and call(ws=BAD) == 3
    for kw in (dict(E=3), dict(N=33), dict(rows=0), dict(n=0), dict(div=0), dict(n_out=-1), dict(n_out=301),
               dict(n=(1 << 24) + 1)):
        assert call(**kw) == 2, kw
    assert call(flags=2) == 1


def test_lora_refusals(L):
    def bank(**kw):
        b = sq.SqLoraBank(S=4, R=16, K=256, N=512, type=sq.SQ_TYPE_BF16, A=1 << 41, B=1 << 41, scale=1 << 41, rank=None)
        for k, v in kw.items():
            setattr(b, k, v)
        return b

    def call(b=None, x=P, M=32, ids=P, off=None, order=None, base=P, ldb=512, y=P, ldy=512, ws=None, wn=0, flags=0):
        b = b or bank()
        return L.sq_lora_add(ctypes.byref(b), x, M, ids, off, order, base, ldb, y, ldy, ws, wn, None, flags, None)
    for kw in (dict(A=None), dict(B=None), dict(scale=None), dict(type=3)):
        assert call(bank(**kw)) == 1, kw
    for kw in (dict(S=0), dict(S=1025), dict(R=0), dict(R=257), dict(K=0), dict(K=65537), dict(N=0)):
        assert call(bank(**kw)) == 2, kw
    for kw in (dict(A=(1 << 41) + 8), dict(rank=(1 << 41) + 4)):
        assert call(bank(**kw)) == 3, kw
    for name in ("x", "ids", "y"):
        assert call(**{name: None}) == 1, name
    assert call(off=P) == 1 and call(order=P) == 1 and call(flags=2) == 1
    assert call(M=0) == 2 and call(M=(1 << 20) + 1) == 2 and call(ldy=511) == 2 and call(ldb=511) == 2
    assert call(ldb=1024, ldy=512) == 1  # in place (base is y) with another row stride
    assert call(x=BAD) == 3 and call(ids=BAD) == 3 and call(y=ctypes.c_void_p((1 << 41) + 2), base=None) == 3
    assert L.sq_lora_workspace_bytes(ctypes.byref(bank()), 64) == 0
    need = L.sq_lora_workspace_bytes(ctypes.byref(bank()), 65)
    assert need >= 65 * 32 * 4 and call(M=65) == 8 and call(M=65, ws=P, wn=need - 1) == 8


def test_combine_refuses_more_columns_than_a_grid_holds(L):
    assert L.sq_combine(P, 8, P, P, 4, 2, 65535 * 256 + 1, None, P, None, 0, None) == 2


def test_grouped_linear_flags(L):
    """SQ_ZERO_REST passes the check of flags (the next one, of alignment, refuses the
    call); bits without a meaning do not."""
    v = _stack(L)

    def call(flags):
        return L.sq_grouped_linear(ctypes.byref(v), 4, 30, P, P, P, P, 2, 8, P, 2, P, 16, P, BAD, 0, None, flags, None)
    assert call(sq.SQ_ZERO_REST) == 3 and call(sq.SQ_ZERO_REST | sq.SQ_LAUNCH_PDL) == 3
    for flags in (sq.SQ_TRUNK_ONLY, 8, 1 << 31):
        assert call(flags) == 1


def _stack_of_arrays(E, N, K, mask, asym):
    """A stack over six host arrays with counting contents (addresses only: no device)."""
    import torch
    rows, cols = E * sq.round_up(N, 16), sq.round_up(K, 128)

    def count(dtype, *shape):
        n = 1
        for s in shape:
            n *= s
        return (torch.arange(n) % 127).to(dtype).reshape(shape)
    arrays = (count(torch.int32, rows, cols // 32), count(torch.float32, rows), count(torch.int8, rows, cols),
              count(torch.float32, rows, cols // 128) + 1, count(torch.int32, rows, cols // 32) + 2 if mask else None,
              count(torch.int32, rows, cols // 128) + 3 if asym else None)
    v = sq.SqPackedWeight()
    v.N, v.K, v.group_size = rows, K, 128
    v.layout = sq.SQ_LAYOUT_TILES_ASYM if asym else sq.SQ_LAYOUT_TILES
    v.sign_stride, v.res_stride, v.scale_stride = cols // 32, cols, cols // 128
    v.sign_bits, v.alpha, v.res_q, v.res_scale, v.mask_bits, v.res_zero = (
        None if t is None else t.data_ptr() for t in arrays)
    return sq.PackedExperts(E, N, K, v, arrays)


@pytest.mark.parametrize("mask,asym", [(0, 0), (1, 0), (0, 1), (1, 1)])
def test_an_expert_of_given_arrays_keeps_them_alive(L, mask, asym):
    """Every address in an expert's view lies in memory that the expert itself holds."""
    import gc
    stack = _stack_of_arrays(3, 30, 300, mask, asym)
    spans = [(t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in stack.keep if t is not None]
    pw = stack.expert(1)
    del stack
    gc.collect()
    held = {pw.sign_bits().data_ptr(), pw.alpha().data_ptr(), pw.res_q().data_ptr(), pw.res_scale().data_ptr()}
    held |= {t.data_ptr() for t in (pw.mask_bits(), pw.res_zero()) if t is not None}
    view = {a for a in (pw.view.sign_bits, pw.view.alpha, pw.view.res_q, pw.view.res_scale, pw.view.mask_bits,
                        pw.view.res_zero) if a}
    assert view == held and len(view) == 4 + mask + asym
    assert all(any(a <= p < b for a, b in spans) for p in view)


@pytest.mark.parametrize("mask,asym", [(0, 0), (1, 1)])
def test_the_arrays_of_an_expert(L, mask, asym):
    """The accessors of an expert show its rows of the stack, and nbytes counts them."""
    import torch
    stack = _stack_of_arrays(3, 30, 300, mask, asym)
    pw, at = stack.expert(2), slice(64, 96)
    sign, alpha, res_q, res_scale, mask_bits, res_zero = stack.keep
    assert torch.equal(pw.sign_bits(), sign[at]) and torch.equal(pw.alpha(), alpha[64:94])
    assert torch.equal(pw.res_q(), res_q[at]) and torch.equal(pw.res_scale(), res_scale[at])
    assert torch.equal(pw.mask_bits(), mask_bits[at]) if mask else pw.mask_bits() is None
    assert torch.equal(pw.res_zero(), res_zero[at]) if asym else pw.res_zero() is None
    assert pw.nbytes * 3 == sum(t.numel() * t.element_size() for t in stack.keep if t is not None)


@pytest.mark.parametrize("layout,mask", [(sq.SQ_LAYOUT_TILES, False), (sq.SQ_LAYOUT_TILES_ASYM, True)])
def test_the_arrays_of_an_expert_of_one_allocation(L, layout, mask):
    import torch
    n = sq.packed_bytes(96, 300, 128, mask, layout)
    buf = torch.zeros(n + 256, dtype=torch.uint8)
    buf = buf[-buf.data_ptr() % 256:][:n]
    stack = sq.PackedExperts(3, 30, 300, sq.SqPackedWeight(), (buf,))
    assert L.sq_packed_view(ctypes.c_void_p(buf.data_ptr()), 96, 300, 128, int(mask), layout, ctypes.byref(stack.view)) == 0
    pw = stack.expert(1)
    v = pw.view
    for t, p, rows in ((pw.sign_bits(), v.sign_bits, 32), (pw.alpha(), v.alpha, 30), (pw.res_q(), v.res_q, 32),
                       (pw.res_scale(), v.res_scale, 32), (pw.mask_bits(), v.mask_bits, 32), (pw.res_zero(), v.res_zero, 32)):
        assert (t is None) == (not p)
        if t is not None:
            assert t.data_ptr() == p and t.shape[0] == rows
    assert pw.buf is stack.keep[0]
    assert pw.nbytes == 32 * (384 + 12 * 4 + 4 + 3 * 4 + (12 * 4 if mask else 0) + (12 if layout == sq.SQ_LAYOUT_TILES_ASYM else 0))


def test_a_sort_workspace_serves_every_shorter_call(L):
    """One allocation for the longest batch: the size does not fall as the batch grows."""
    for k in (1, 2, 3, 5, 7, 8, 12, 31, 32):
        for E in (32, 33, 128, 1024):
            longest = 0
            for T in sorted({*range(1, 700), *range(700, 9000, 7), *range(9000, (1 << 24) // k, 40009), (1 << 24) // k}):
                need = L.sq_route_workspace_bytes(T, E, k)
                assert need >= longest, (T, E, k)
                longest = need
    longest = 0
    for n in sorted({*range(4000, 140000, 11), *range(140000, 1 << 24, 9973), 1 << 24}):
        need = L.sq_segment_workspace_bytes(n, 77)
        assert need >= longest, n
        longest = need


def test_an_adapter_workspace_serves_every_shorter_call(L):
    for S, R in ((1, 8), (77, 33), (1024, 256)):
        b = sq.SqLoraBank(S=S, R=R, K=256, N=512, type=sq.SQ_TYPE_BF16, A=1 << 41, B=1 << 41, scale=1 << 41, rank=None)
        longest = 0
        for M in (*range(1, 6000, 3), *range(6000, 1 << 20, 1013), 1 << 20):
            need = L.sq_lora_workspace_bytes(ctypes.byref(b), M)
            assert need >= longest, (S, R, M)
            longest = need


def _no_device(rc):
    """Past every check of arguments: no usable device here, or (on one) not launched."""
    return rc not in (0, 1, 2, 3, 8)


def _at(words):
    return ctypes.c_void_p((1 << 41) + 4 * words)


@pytest.fixture
def no_gpu():
    import torch
    if torch.cuda.is_available():
        pytest.skip("these calls would be launched on made-up addresses")


def test_combine_refuses_a_result_over_its_inputs(L, no_gpu):
    far = _at(1 << 30)

    def call(z=_at(0), rows=8, T=4, N=64, base=None, out=far):
        return L.sq_combine(z, rows, P, P, T, 2, N, base, out, None, 0, None)
    assert _no_device(call()) and _no_device(call(base=far))
    # z holds words [0, 512), out 256 words
    assert call(out=_at(0)) == 1 and call(out=_at(508)) == 1 and _no_device(call(out=_at(512)))
    assert call(z=_at(252), out=_at(0)) == 1 and _no_device(call(z=_at(256), out=_at(0)))
    # base: out itself or apart
    at = 1 << 30
    assert call(base=_at(at + 252)) == 1 and call(base=_at(at - 252)) == 1
    assert _no_device(call(base=_at(at + 256))) and _no_device(call(base=_at(at - 256)))


def test_lora_refuses_a_result_over_its_inputs(L, no_gpu):
    b = sq.SqLoraBank(S=4, R=16, K=256, N=100, type=sq.SQ_TYPE_BF16, A=1 << 45, B=1 << 45, scale=1 << 45, rank=None)

    def call(x=_at(1 << 32), M=32, base=None, ldb=512, y=_at(1 << 30), ldy=512):
        return L.sq_lora_add(ctypes.byref(b), x, M, P, None, None, base, ldb, y, ldy, None, 0, None, 0, None)
    o = 1 << 30
    assert _no_device(call()) and _no_device(call(base=_at(o)))
    # column slices of one matrix of 512: side by side or over one another, from any row on
    for col, bad in ((99, 1), (100, 0), (412, 0), (413, 1), (-99, 1), (-100, 0), (512, 1), (-512, 1), (512 * 31 + 50, 1),
                     (512 * 31 + 100, 0), (512 * 32, 0), (-512 * 31 - 99, 1), (-512 * 32, 0), (512 * 7 + 300, 0)):
        rc = call(base=_at(o + col))
        assert (rc == 1) if bad else _no_device(rc), col
    # other strides: found wherever two rows meet
    assert call(base=_at(o + 100), ldb=511) == 1 and _no_device(call(base=_at(o + 200), ldb=513, M=3))
    assert call(base=_at(o + 200), ldb=800, M=3) == 1  # 1000 .. 1099 and 1024 .. 1123
    assert _no_device(call(base=_at(o + 100), y=_at(o), M=1, ldb=100, ldy=100)) and call(base=_at(o + 99), M=1, ldb=100) == 1
    # x: rows of 256
    assert call(x=_at(o)) == 1 and call(x=_at(o + 32 * 512 - 512 + 96)) == 1 and call(x=_at(o - 32 * 256 + 4)) == 1
    assert _no_device(call(x=_at(o - 32 * 256))) and _no_device(call(x=_at(o + 31 * 512 + 100)))
    # ... each row of y within the same row of x
    assert _no_device(call(x=_at(o), ldy=256)) and call(x=_at(o + 4), ldy=256) == 1
    assert _no_device(call(x=_at(o - 156), ldy=256)) and call(x=_at(o - 160), ldy=256) == 1
    assert _no_device(call(x=_at(o + 4), M=1)) and call(x=_at(o - 156), ldy=512) == 1


def test_rows_that_overlap_are_found_as_by_listing_them(L, no_gpu):
    """Small strides against a set of every word."""
    import itertools
    import random
    rng = random.Random(1)
    for _ in range(400):
        N, M = rng.randint(1, 6), rng.randint(1, 6)
        lda, ldb, off = rng.randint(N, 12), rng.randint(N, 12), rng.randint(-40, 40)
        b = sq.SqLoraBank(S=1, R=1, K=1, N=N, type=sq.SQ_TYPE_F32, A=1 << 45, B=1 << 45, scale=1 << 45, rank=None)
        o = 1 << 30
        if off == 0 and lda != ldb:
            continue  # (refused for its strides)
        rows = [{o + i * lda + c for i, c in itertools.product(range(M), range(N))},
                {o + off + i * ldb + c for i, c in itertools.product(range(M), range(N))}]
        rc = L.sq_lora_add(ctypes.byref(b), _at(1 << 33), M, P, None, None, _at(o + off), ldb, _at(o), lda, None, 0, None,
                           0, None)
        bad = off != 0 and bool(rows[0] & rows[1])
        assert (rc == 1) if bad else _no_device(rc), (N, M, lda, ldb, off)
