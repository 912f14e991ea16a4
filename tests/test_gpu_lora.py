"""Low-rank adapters of many requests against plain numpy in 64 bits.

Tolerance, from the arithmetic: v = A x is a sum of K binary32 products in at
most K/32 + 64 roundings along any one path (on the tensor cores ceil(K/32)/16
steps of two k16 products of up to six parts, then 16 slices; fewer on the CUDA
cores), the sum over the rank at most R + 32, each rounding at most 2^-23 of the
sum of magnitudes (a tensor-core addition may truncate), the cut of a value
into parts 2^-23 of it, and the last addition 2^-24 of |y|:
  |error| <= 2^-23 ((K/32 + 64) + (R + 32)) scale sum_r |B_nr| sum_k |A_rk x_k| + 2^-23 |y|.
"""
import numpy as np
import pytest
import torch

import decode_matvec_sq_b200 as sq

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def built(cuda_device):
    from decode_matvec_sq_b200 import build
    build.build_all()
    sq.device_check()
    yield


class Case:
    def __init__(self, M, S, R, K, N, dtype, none=0.2, ragged=True, seed=0, x_scale=1.0, ids=None):
        rng = np.random.default_rng(seed + M + 3 * S + 5 * R + 7 * K + 11 * N)
        self.M, self.S, self.R, self.K, self.N = M, S, R, K, N
        self.rank = rng.integers(0, R + 1, S).astype(np.int32) if ragged else np.full(S, R, np.int32)
        A = torch.from_numpy((rng.standard_normal((S, R, K)) / np.sqrt(K)).astype(np.float32)).to(TYPES[dtype])
        B = torch.from_numpy((0.05 * rng.standard_normal((S, N, R))).astype(np.float32)).to(TYPES[dtype])
        self.A, self.B = A.double().numpy(), B.double().numpy()
        for a in range(S):  # what lies past an adapter's rank is not used, whatever it holds
            A[a, self.rank[a]:] = float("nan")
            B[a, :, self.rank[a]:] = float("nan")
        self.scale = (0.5 + rng.random(S)).astype(np.float32)
        self.ids = np.where(rng.random(M) < none, -1, rng.integers(0, S, M)).astype(np.int32) if ids is None else ids
        self.x = (x_scale * rng.standard_normal((M, K))).astype(np.float32)
        self.base = rng.standard_normal((M, N)).astype(np.float32)
        dev = [torch.from_numpy(v).cuda() for v in (self.scale, self.rank, self.x, self.ids, self.base)]
        self.bank = sq.LoraBank(A.cuda(), B.cuda(), dev[0], dev[1])
        self.xd, self.idsd, self.based = dev[2:]
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def want(self, base=True):
        y = self.base.astype(np.float64) if base else np.zeros((self.M, self.N))
        tol = np.zeros_like(y)
        c = (self.K / 32 + 64 + self.R + 32) * 2.0 ** -23
        for a in range(self.S):
            t, r = np.flatnonzero(self.ids == a), self.rank[a]
            A, B, s, x = self.A[a, :r], self.B[a, :, :r], float(self.scale[a]), self.x[t].astype(np.float64)
            y[t] += s * (x @ A.T) @ B.T
            tol[t] += c * s * (np.abs(x) @ np.abs(A).T) @ np.abs(B).T
        return y, tol + 2.0 ** -23 * np.abs(y)

    def check(self, y, base=True, rows=None):
        torch.cuda.synchronize()
        want, tol = self.want(base)
        rows = slice(None) if rows is None else rows
        err = np.abs(y.cpu().numpy().astype(np.float64) - want)[rows]
        assert np.all(err <= tol[rows]), float(np.nanmax(err / np.maximum(tol[rows], 1e-300)))

    def run(self, **kw):
        kw.setdefault("base", self.based)
        return sq.lora_add(self.bank, self.xd, self.idsd, status=self.status, **kw)


SHAPES = [(1, 1, 1, 1, 1), (1, 8, 16, 4096, 4096), (3, 2, 8, 100, 37), (64, 5, 64, 512, 1000), (17, 40, 24, 1000, 520),
          (64, 3, 256, 300, 300), (65, 4, 8, 129, 64), (200, 7, 33, 1003, 1001), (333, 5, 24, 2048, 520),
          (700, 50, 100, 264, 136), (130, 2, 256, 640, 72), (1500, 8, 64, 1024, 1088)]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("M,S,R,K,N", SHAPES)
def test_lora(M, S, R, K, N, dtype):
    c = Case(M, S, R, K, N, dtype)
    c.check(c.run())
    assert c.status.item() == 0


@pytest.mark.parametrize("M", [5, 300])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_full_rank_without_a_rank_array(M, dtype):
    c = Case(M, 3, 16, 256, 200, dtype, ragged=False)
    c.bank = sq.LoraBank(c.bank.A, c.bank.B, c.bank.scale)
    c.check(c.run())


@pytest.mark.parametrize("M", [6, 300])
def test_without_a_base(M):
    c = Case(M, 3, 16, 256, 200, "bf16")
    c.check(c.run(base=None), base=False)


@pytest.mark.parametrize("M", [10, 64, 65, 400])
@pytest.mark.parametrize("col,ld", [(128, 512), (3, 301)])
def test_in_place_on_a_slice(M, col, ld):
    """y is base is a column slice of a wider projection: nothing else changes,
    and rows without an adapter keep their bits."""
    c = Case(M, 4, 20, 192, 200, "f16", none=0.4)
    wide = torch.randn(M, ld, device="cuda")
    part = wide[:, col:col + 200]
    part.copy_(c.based)
    before = wide.clone()
    y = c.run(base=part, y=part)
    c.check(y)
    outside = torch.ones(ld, dtype=torch.bool, device="cuda")
    outside[col:col + 200] = False
    assert torch.equal(wide[:, outside], before[:, outside])
    none = torch.from_numpy(c.ids).cuda() < 0
    assert torch.equal(wide[none], before[none])


@pytest.mark.parametrize("M", [20, 300])
def test_rows_without_adapter_copy_the_base(M):
    c = Case(M, 4, 8, 64, 100, "bf16", none=1.0)
    assert torch.equal(c.run(), c.based)
    assert torch.equal(c.run(base=None), torch.zeros_like(c.based))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("x_scale", [1e-30, 1e-6, 1e6, 1e30])
def test_scales_of_the_activations(x_scale, dtype):
    """The parts of a value keep its range."""
    c = Case(200, 3, 24, 256, 128, dtype, x_scale=x_scale)
    c.base[:] = 0
    c.based.zero_()
    c.check(c.run())


@pytest.mark.parametrize("M", [12, 200])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("value", [float("inf"), float("nan"), -float("inf")])
def test_a_token_that_is_not_finite_touches_no_other(M, dtype, value):
    c = Case(M, 2, 16, 128, 96, dtype, none=0.0, ragged=False)
    c.xd[7, 5] = value
    y = c.run()
    torch.cuda.synchronize()
    assert c.status.item() == sq.STATUS_CODE["SQ_ERR_NONFINITE"]
    assert not torch.isfinite(y[7]).any()
    c.check(y, rows=np.arange(M) != 7)


@pytest.mark.parametrize("M", [12, 200])
def test_ids_out_of_range_have_no_adapter(M):
    c = Case(M, 3, 16, 128, 96, "bf16")
    c.idsd[[1, 4]] = torch.tensor([3, -2], dtype=torch.int32, device="cuda")
    c.ids[[1, 4]] = -1
    y = c.run()
    c.check(y)
    assert c.status.item() == sq.STATUS_CODE["SQ_ERR_INVALID_ARG"]


@pytest.mark.parametrize("M", [40, 1000])
def test_one_sort_serves_several_projections(M):
    c, d = Case(M, 6, 16, 256, 512, "bf16", seed=1), Case(M, 6, 8, 256, 128, "f16", seed=2)
    d.ids, d.idsd = c.ids, c.idsd
    seg = sq.segment(c.idsd, 6)
    c.check(c.run(segments=seg))
    d.check(d.run(segments=seg))
    assert torch.equal(c.run(segments=seg), c.run())


@pytest.mark.parametrize("M", [64, 300])
def test_same_call_twice_gives_the_same_bits(M):
    c = Case(M, 6, 32, 1024, 512, "bf16")
    assert torch.equal(c.run(), c.run())


@pytest.mark.parametrize("M", [32, 500])
def test_replayed_graph_follows_the_ids(M):
    c = Case(M, 5, 16, 256, 320, "bf16")
    ws = sq.new_lora_workspace(c.bank, M)
    c.run(workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = c.run(workspace=ws, pdl=True)
    rng = np.random.default_rng(3)
    for hi in (5, 1, 3):
        c.ids = rng.integers(-1, hi, M).astype(np.int32)
        c.idsd.copy_(torch.from_numpy(c.ids))
        torch.cuda.synchronize()
        g.replay()
        c.check(y)


def test_calls_on_two_streams():
    a, b = Case(400, 3, 16, 512, 640, "bf16", seed=1), Case(64, 8, 32, 300, 1000, "f32", seed=2)
    wa = sq.new_lora_workspace(a.bank, a.M)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    ys = []
    for _ in range(4):
        with torch.cuda.stream(s1):
            ys.append((a, a.run(workspace=wa)))
        with torch.cuda.stream(s2):
            ys.append((b, b.run()))
    torch.cuda.synchronize()
    for c, y in ys:
        c.check(y)


def test_dependent_launches_back_to_back_share_a_workspace():
    """Projections of one step in stream order on one workspace, each launched
    before the one ahead of it has ended."""
    cs = [Case(300, 4, 16, 256, 256, "bf16", seed=s) for s in range(3)]
    ws = sq.new_lora_workspace(cs[0].bank, 300)
    torch.cuda.synchronize()
    ys = [c.run(workspace=ws, pdl=True) for c in cs for _ in range(3)]
    torch.cuda.synchronize()
    for i, y in enumerate(ys):
        cs[i // 3].check(y)


def test_beside_the_shared_projection():
    """The decode linear layer and its adapters as a serving step runs them."""
    import oracle
    M, K, N = 9, 512, 768
    c = Case(M, 4, 16, K, N, "bf16")
    rng = np.random.default_rng(4)
    W = rng.laplace(0, 0.02, (N, K)).astype(np.float32)
    idx = np.array([3, 77], np.int32)
    idxd = torch.from_numpy(idx).cuda()
    pw = sq.decompose_pack(torch.from_numpy(W).cuda())
    y = sq.quantize_linear(pw, c.xd, idxd, status=c.status)
    sq.lora_add(c.bank, c.xd, c.idsd, y, y=y, status=c.status, pdl=True)
    torch.cuda.synchronize()
    assert c.status.item() == 0
    ref = oracle.linear(oracle.decompose(W), *oracle.quantize_act(c.x, idx), idx)
    c.base = ref
    want, tol = c.want()
    assert (np.abs(y.cpu().numpy() - want) <= tol + 1e-5 * oracle.abs_dot(W, c.x)).all()


@pytest.mark.parametrize("M", [1 << 20, (1 << 20) - 7])
def test_the_most_tokens(M):
    """More 16-token groups than a grid has rows.  Small integers: every sum is exact."""
    S, R, K, N = 3, 2, 8, 4
    g = torch.Generator(device="cuda").manual_seed(M)
    rnd = lambda *s: torch.randint(-3, 4, s, generator=g, device="cuda").float()
    bank = sq.LoraBank(rnd(S, R, K), rnd(S, N, R), torch.tensor([1.0, 2.0, 0.5], device="cuda"))
    x, base = rnd(M, K), rnd(M, N)
    ids = torch.randint(-1, S, (M,), generator=g, device="cuda", dtype=torch.int32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = sq.lora_add(bank, x, ids, base=base, status=st)
    at = ids.clamp(min=0).long()
    v = (bank.A[at] * x[:, None, :]).sum(2) * bank.scale[at][:, None]
    want = base + torch.where(ids[:, None] >= 0, (bank.B[at] * v[:, None, :]).sum(2), 0.0)
    assert st.item() == 0 and torch.equal(y, want)


@pytest.mark.parametrize("M,S", [(65, 1), (65, 1024), (300, 1023), (511, 40), (512, 1), (512, 1024), (513, 1024)])
def test_a_sort_of_ones_own_gives_the_same_bits(M, S):
    """The call's own sort (by launch or within the kernels) against segments()."""
    c = Case(M, S, 16, 264, 72, "bf16")
    y = c.run()
    c.check(y)
    z = c.run(segments=sq.segment(c.idsd, S))
    assert torch.equal(y, z) and c.status.item() == 0


@pytest.mark.parametrize("M", [100, 512, 600])
def test_no_token_has_an_adapter(M):
    c = Case(M, 3, 16, 264, 72, "f16")
    c.idsd.fill_(-1)
    assert torch.equal(c.run(), c.based) and c.status.item() == 0
