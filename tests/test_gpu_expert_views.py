"""An expert of a stack used as a weight of its own after the stack is gone."""
import gc

import numpy as np
import pytest
import torch

import decode_matvec_sq_b200 as sq
import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built(cuda_device):
    from decode_matvec_sq_b200 import build
    build.build_all()
    sq.device_check()
    yield


@pytest.mark.parametrize("from_arrays", [False, True])
def test_an_expert_outlives_its_stack(from_arrays):
    """Memory freed with the stack would be overwritten by the blocks allocated next."""
    N, K = 50, 300
    rng = np.random.default_rng(1)
    W = rng.laplace(0, 0.02, (2, N, K)).astype(np.float32)
    stack = sq.alloc_experts(2, N, K, with_mask=True)
    for e in range(2):
        sq.decompose_pack(torch.from_numpy(W[e]).cuda(), trunk_percent=60, out=stack.expert(e))
    if from_arrays:
        parts = [stack.expert(e) for e in range(2)]

        def both(name):
            return torch.cat([getattr(p, name)() for p in parts]).contiguous()
        alpha = torch.cat([p.arrays["alpha"] for p in parts])
        stack = sq.experts_from_arrays(2, N, K, both("sign_bits"), alpha, both("res_q"), both("res_scale"),
                                       mask_bits=both("mask_bits"))
        del parts, alpha
    pw = stack.expert(1)
    torch.cuda.synchronize()
    del stack
    gc.collect()
    junk = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in (512, 2048, 4096, 8192, 32768, 65536) for _ in range(8)]
    x = rng.standard_normal((3, K)).astype(np.float32)
    idx = np.array([4], np.int32)
    idxd = torch.from_numpy(idx).cuda()
    y = sq.linear(pw, *sq.quantize_act(torch.from_numpy(x).cuda(), idxd), idxd).cpu().numpy()
    ref = oracle.linear(oracle.decompose(W[1], P=60), *oracle.quantize_act(x, idx), idx)
    assert len(junk) == 48 and (np.abs(y - ref) <= 1e-5 * oracle.abs_dot(W[1], x)).all()
    assert pw.nbytes == sum(t.numel() * t.element_size() for t in pw.arrays.values())
