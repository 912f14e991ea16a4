"""The linear layer grouped by expert against the 64-bit oracle of the linear
layer, expert by expert: y within 1e-5 * sum_j |W_rj x_j|, the bound every
decode and prefill kernel of one weight is held to (the longest binary32 chain
here, K = 14336, has 112 groups: 112 * 2^-24 = 6.7e-6 of the sum of magnitudes)."""
import ctypes

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


class Case:
    """E experts, activations of `rows` rows, and a sort of entries with the
    given counts per expert; entry i's row is order[i] // div."""

    def __init__(self, E, N, K, counts, layout=sq.SQ_LAYOUT_TILES, P=-1, n_out=5, div=2, spare=0, seed=0, by_place=False):
        rng = np.random.default_rng(seed + E + 3 * N + 7 * K)
        self.E, self.N, self.K, self.P, self.layout, self.div = E, N, K, P, layout, div
        self.W = rng.laplace(0, 0.02, (E, N, K)).astype(np.float32)
        self.experts = sq.alloc_experts(E, N, K, with_mask=P > 0, layout=layout)
        for e in range(E):
            sq.decompose_pack(torch.from_numpy(self.W[e]).cuda(), trunk_percent=P, out=self.experts.expert(e))
        live = int(sum(counts))
        self.n = live + spare
        self.offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        if by_place:
            self.rows, self.order = self.n, None
            self.src = np.arange(self.n)
        else:
            self.rows = max(1, -(-self.n // div))
            order = rng.permutation(self.rows * div)[:self.n].astype(np.int32)
            order[live:] = -1
            self.order, self.src = order, order // div
        self.x = rng.standard_normal((self.rows, K)).astype(np.float32)
        self.idx = np.sort(rng.choice(K, min(n_out, K), replace=False)).astype(np.int32)
        self.x[:, self.idx] *= 30.0
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.idxd = torch.from_numpy(self.idx).cuda()
        self.xq, self.sx, self.xo = sq.quantize_act(torch.from_numpy(self.x).cuda(), self.idxd, status=self.status)
        self.offd = torch.from_numpy(self.offsets).cuda()
        self.ordd = None if self.order is None else torch.from_numpy(self.order).cuda()

    def run(self, **kw):
        y = torch.full((self.n, self.N), 12345.0, device="cuda")
        return sq.grouped_linear(self.experts, self.xq, self.sx, self.xo, self.idxd, self.offd, order=self.ordd,
                                 div=self.div if self.order is not None else 1, y=y, status=self.status, **kw)

    def check(self, y):
        torch.cuda.synchronize()
        assert self.status.item() == 0
        y = y.cpu().numpy().astype(np.float64)
        for e in range(self.E):
            a, b = self.offsets[e], self.offsets[e + 1]
            if a == b:
                continue
            W = self.W[e]
            if self.layout == sq.SQ_LAYOUT_TILES_ASYM:
                d, fn = oracle.decompose_asym(W, P=self.P), oracle.linear_asym
            else:
                d, fn = oracle.decompose(W, P=self.P), oracle.linear
            x = self.x[self.src[a:b]]
            oxq, osx, oxo = oracle.quantize_act(x, self.idx)
            ref, bound = fn(d, oxq, osx, oxo, self.idx), oracle.abs_dot(W, x)
            err = np.abs(y[a:b] - ref)
            assert np.all(err <= TOL * bound), (e, float((err / bound).max()))
        assert (y[self.offsets[-1]:] == 12345.0).all()  # rows behind the last segment


@pytest.mark.parametrize("layout", [sq.SQ_LAYOUT_TILES, sq.SQ_LAYOUT_TILES_ASYM])
@pytest.mark.parametrize("P", [-1, 60])
@pytest.mark.parametrize("N,K,counts", [
    (1, 1, [1]), (16, 128, [0, 1, 0]), (40, 300, [3, 0, 9, 1]), (513, 1000, [8, 17, 0, 16, 1]),
    (33, 129, [40, 0, 0, 5]), (64, 4096, [1, 1]), (24, 2050, [7, 30]), (200, 257, [0, 130, 64, 3])])
def test_grouped_linear(layout, P, N, K, counts):
    c = Case(len(counts), N, K, counts, layout, P, n_out=min(9, K), spare=3)
    c.check(c.run())


@pytest.mark.parametrize("n_out", [0, 1, 64])
@pytest.mark.parametrize("by_place", [False, True])
def test_outliers_and_rows_in_place_order(n_out, by_place):
    c = Case(4, 100, 640, [5, 0, 21, 2], n_out=n_out, by_place=by_place)
    c.check(c.run())


@pytest.mark.parametrize("counts", [[1, 0, 1, 0], [0, 0, 0, 300], [20, 150, 3, 257]])
def test_wide_experts(counts):
    """Row blocks and channel groups spread over every CTA and warp."""
    c = Case(4, 1500, 2816, counts, n_out=14, seed=3)
    c.check(c.run())


def test_all_tokens_drop():
    c = Case(3, 64, 256, [0, 0, 0], spare=5)
    c.check(c.run())


def test_every_outlier_channel_in_one_group():
    c = Case(2, 48, 512, [3, 2], n_out=5)
    c.idx = np.arange(130, 135, dtype=np.int32)
    c.idxd = torch.from_numpy(c.idx).cuda()
    c.xq, c.sx, c.xo = sq.quantize_act(torch.from_numpy(c.x).cuda(), c.idxd)
    c.check(c.run())


def test_expert_view_equals_the_linear_layer_of_one_weight():
    c = Case(3, 100, 512, [2, 2, 2], by_place=True)
    y = c.run()
    for e in range(3):
        part = [v[2 * e:2 * e + 2].clone() for v in (c.xq, c.sx, c.xo)]  # (16-byte aligned copies)
        ref = sq.linear(c.experts.expert(e), *part, c.idxd)
        bound = torch.from_numpy(oracle.abs_dot(c.W[e], c.x[2 * e:2 * e + 2])).cuda()
        assert ((y[2 * e:2 * e + 2] - ref).abs() <= 2 * TOL * bound).all()


def test_experts_from_arrays_uses_the_arrays_in_place():
    c = Case(2, 30, 300, [4, 3], P=60)
    v, rows, cols = c.experts.view, 2 * 32, 384
    buf, base = c.experts.keep[0], c.experts.keep[0].data_ptr()

    def arr(p, dtype, shape):
        n = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        return buf[p - base:p - base + n].view(dtype).view(*shape).clone()
    c.experts = sq.experts_from_arrays(
        2, 30, 300, arr(v.sign_bits, torch.int32, (rows, cols // 32)), arr(v.alpha, torch.float32, (rows,)),
        arr(v.res_q, torch.int8, (rows, cols)), arr(v.res_scale, torch.float32, (rows, cols // 128)),
        mask_bits=arr(v.mask_bits, torch.int32, (rows, cols // 32)))
    c.check(c.run())


def test_replayed_graph_follows_the_route():
    """One captured call (dependent launches), replayed on other counts."""
    c = Case(4, 96, 384, [10, 0, 7, 3], spare=12)
    c.run()
    torch.cuda.synchronize()
    ws = sq.new_grouped_workspace(c.experts, c.n)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = c.run(workspace=ws, pdl=True)
    rng = np.random.default_rng(5)
    for counts in ([10, 0, 7, 3], [0, 20, 0, 0], [1, 1, 1, 1], [0, 0, 0, 32]):
        c.offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        order = rng.permutation(c.rows * c.div)[:c.n].astype(np.int32)
        order[c.offsets[-1]:] = -1
        c.src = order // c.div
        c.offd.copy_(torch.from_numpy(c.offsets))
        c.ordd.copy_(torch.from_numpy(order))
        torch.cuda.synchronize()
        g.replay()
        c.check(y)


def test_calls_on_two_streams():
    a, b = Case(3, 200, 512, [40, 30, 50], seed=1), Case(2, 300, 640, [20, 90], seed=2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    wa, wb = sq.new_grouped_workspace(a.experts, a.n), sq.new_grouped_workspace(b.experts, b.n)
    torch.cuda.synchronize()
    ys = []
    for _ in range(4):
        with torch.cuda.stream(s1):
            ya = a.run(workspace=wa)
        with torch.cuda.stream(s2):
            yb = b.run(workspace=wb)
        ys += [(a, ya), (b, yb)]
    torch.cuda.synchronize()
    for c, y in ys:
        c.check(y)


def test_same_call_twice_gives_the_same_bits():
    c = Case(5, 300, 1000, [33, 2, 0, 70, 9])
    assert torch.equal(c.run(), c.run())


@pytest.mark.parametrize("what", ["descending", "past_n", "negative", "order", "order_negative", "idx"])
def test_bad_device_arrays_are_reported(what):
    """The kernels' own bounds checks turn each into a status."""
    c = Case(3, 64, 256, [4, 4, 4])
    torch.cuda.synchronize()
    if what == "descending":
        c.offd.copy_(torch.tensor([0, 8, 4, 12]))
    elif what == "past_n":
        c.offd.copy_(torch.tensor([0, 4, 8, 1 << 30]))
    elif what == "negative":
        c.offd.copy_(torch.tensor([-5, 4, 8, 12]))
    elif what == "order":
        c.ordd[3] = c.rows * c.div
    elif what == "order_negative":
        c.ordd[3] = -1
    else:
        c.idxd.copy_(torch.tensor([1, 5, 5, 9, 300]))
    c.run()
    torch.cuda.synchronize()
    assert c.status.item() == sq.STATUS_CODE["SQ_ERR_INVALID_ARG"]


def test_a_layer_of_experts_end_to_end():
    """Router, up projection, activation, down projection and combine, as a
    serving step runs them, against the same computed expert by expert in 64 bits
    from the same routes and the same quantized activations."""
    T, E, k, D, H = 37, 6, 2, 256, 384
    rng = np.random.default_rng(9)
    W1 = rng.laplace(0, 0.05, (E, H, D)).astype(np.float32)
    W2 = rng.laplace(0, 0.05, (E, D, H)).astype(np.float32)
    up, down = sq.alloc_experts(E, H, D), sq.alloc_experts(E, D, H)
    for e in range(E):
        sq.decompose_pack(torch.from_numpy(W1[e]).cuda(), out=up.expert(e))
        sq.decompose_pack(torch.from_numpy(W2[e]).cuda(), out=down.expert(e))
    x = torch.from_numpy(rng.standard_normal((T, D)).astype(np.float32)).cuda()
    logits = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)).cuda()
    idx1 = torch.tensor([3, 200], dtype=torch.int32, device="cuda")
    idx2 = torch.tensor([7], dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    r = sq.route(logits, k, status=st)
    q1 = sq.quantize_act(x, idx1, status=st)
    h = sq.grouped_linear(up, *q1, idx1, r.offsets, order=r.order, div=k, status=st)
    h = torch.nn.functional.silu(h)
    q2 = sq.quantize_act(h, idx2, status=st)
    z = sq.grouped_linear(down, *q2, idx2, r.offsets, status=st)
    out = sq.combine(z, r.gates, r.place, base=x, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    i1, i2 = idx1.cpu().numpy(), idx2.cpu().numpy()
    ids, gates, place = r.ids.cpu().numpy(), r.gates.cpu().numpy().astype(np.float64), r.place.cpu().numpy()
    d2 = [oracle.decompose(W2[e]) for e in range(E)]
    hh, want, mag = h.cpu().numpy(), x.cpu().numpy().astype(np.float64), np.abs(x.cpu().numpy()).astype(np.float64)
    for t in range(T):
        for j in range(k):
            hp = hh[place[t, j]][None]
            ref = oracle.linear(d2[ids[t, j]], *oracle.quantize_act(hp, i2), i2)[0]
            want[t] += gates[t, j] * ref
            mag[t] += gates[t, j] * oracle.abs_dot(W2[ids[t, j]], hp)[0]
    assert (np.abs(out.cpu().numpy() - want) <= 2 * TOL * mag).all()


# ---- many tokens per expert (the tcgen05 kernel: 24 entries per expert and more) -----
# Outlier products there are sums of tf32 parts that miss 2^-21 of each product and may
# truncate 2^-23 of a sum of 24 terms per addition: 2e-6 of the sum of magnitudes, within TOL.
@pytest.mark.parametrize("P", [-1, 60])
@pytest.mark.parametrize("n_out", [1, 15, 16, 17, 33, 100, 128, 129])
def test_outlier_chunks_with_many_tokens(n_out, P):
    c = Case(3, 200, 1000, [170, 0, 33], P=P, n_out=n_out)
    c.check(c.run())


@pytest.mark.parametrize("N,K,counts,div", [
    (1, 1, [321], 1), (17, 128, [161, 1, 480], 3), (129, 129, [31, 33, 160, 0], 5), (300, 384, [1, 700, 0, 0, 2], 7),
    (4090, 256, [100, 3], 2)])
def test_tiles_of_many_tokens(N, K, counts, div):
    """Tokens just around a tile's 160, one channel group per tile, rows past a tile's 128."""
    c = Case(len(counts), N, K, counts, n_out=min(K, 3), div=div, spare=2)
    c.check(c.run())


def test_outliers_crowded_into_one_group_with_many_tokens():
    c = Case(2, 260, 512, [60, 170], n_out=40)
    c.idx = np.arange(250, 290, dtype=np.int32)
    c.idxd = torch.from_numpy(c.idx).cuda()
    c.xq, c.sx, c.xo = sq.quantize_act(torch.from_numpy(c.x).cuda(), c.idxd)
    c.check(c.run())


@pytest.mark.parametrize("E,per", [(33, 1), (40, 30), (1024, 1), (1024, 25)])
def test_many_experts(E, per):
    """More experts than a warp's lanes, up to the largest stack, in both kernels."""
    rng = np.random.default_rng(E + per)
    counts = rng.multinomial(E * per, rng.dirichlet(np.full(E, 0.3))).tolist()
    c = Case(E, 24, 200, counts, n_out=2, spare=1)
    c.check(c.run())


@pytest.mark.parametrize("per", [2, 60])
def test_an_entry_that_occurs_twice(per):
    c = Case(3, 100, 300, [per, per, per])
    order = c.order.copy()
    order[per:2 * per] = order[:per]  # the same rows at two experts
    order[1] = order[0]               # and twice at one
    c.src = order // c.div
    c.ordd.copy_(torch.from_numpy(order))
    c.check(c.run())


@pytest.mark.parametrize("counts", [[2, 3], [60, 70]])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_row_that_is_not_finite_touches_no_other(counts, value):
    c = Case(2, 150, 400, counts, n_out=3, div=1)
    y = c.run()
    c.check(y)
    row = int(c.src[1])
    x = torch.from_numpy(c.x).cuda()
    x[row, 5] = value
    x[row, int(c.idx[0])] = value
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.xq, c.sx, c.xo = sq.quantize_act(x, c.idxd, status=st)
    z = c.run()
    other = torch.arange(c.n, device="cuda") != 1
    assert torch.equal(y[other], z[other])


@pytest.mark.parametrize("what", ["descending", "past_n", "negative", "order", "order_negative", "idx", "idx_past_k"])
def test_bad_device_arrays_are_reported_with_many_tokens(what):
    c = Case(3, 140, 256, [40, 170, 30])
    n = c.n
    torch.cuda.synchronize()
    if what == "descending":
        c.offd.copy_(torch.tensor([0, 200, 40, n]))
    elif what == "past_n":
        c.offd.copy_(torch.tensor([0, 40, 210, 1 << 30]))
    elif what == "negative":
        c.offd.copy_(torch.tensor([-5, 40, 210, n]))
    elif what == "order":
        c.ordd[3] = c.rows * c.div
    elif what == "order_negative":
        c.ordd[3] = -1
    elif what == "idx":
        c.idxd.copy_(torch.tensor([1, 5, 5, 9, 200]))
    else:
        c.idxd.copy_(torch.tensor([1, 5, 6, 9, 256]))
    c.run()
    torch.cuda.synchronize()
    assert c.status.item() == sq.STATUS_CODE["SQ_ERR_INVALID_ARG"]


def test_a_captured_call_with_many_tokens_follows_the_route():
    """Captured once with its workspace, beside eager calls between the replays."""
    c = Case(3, 96, 384, [100, 0, 7], spare=60, n_out=20)
    ws = sq.new_grouped_workspace(c.experts, c.n)
    c.run(workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = c.run(workspace=ws, pdl=True)
    rng = np.random.default_rng(6)
    for counts in ([100, 0, 7], [0, 167, 0], [1, 1, 1], [0, 0, 0], [50, 50, 67]):
        c.offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        order = rng.permutation(c.rows * c.div)[:c.n].astype(np.int32)
        order[c.offsets[-1]:] = -1
        c.src = order // c.div
        c.offd.copy_(torch.from_numpy(c.offsets))
        c.ordd.copy_(torch.from_numpy(order))
        y.fill_(12345.0)
        torch.cuda.synchronize()
        g.replay()
        c.check(y)
        c.check(c.run())
