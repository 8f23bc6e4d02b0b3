"""Slots without an expert (id -1, what moe_route gives where nothing is left to select) in the
routed products."""
import numpy as np
import pytest
import torch

import fp16_gemm_b200 as sp
import synth
from helpers import to_dev
from test_parity_moe_block import _device_ops

pytestmark = pytest.mark.gpu


def _block(sparse, dtype, T=40, topk=3):
    d = synth.moe_block(seed=41, E=4, H=512, F=512, T=T, topk=topk)
    x = to_dev(d["X"], "bf16").to(dtype)
    return x, torch.from_numpy(d["routing"]).cuda(), torch.from_numpy(d["router_w"]).cuda(), _device_ops(d, sparse, sparse)


@pytest.mark.parametrize("bad", [-1, 4, 2**31 - 1])
@pytest.mark.parametrize("weight", [0.0, 0.5, float("nan")])
@pytest.mark.parametrize("sparse", [False, True], ids=["dense", "sparse24"])
def test_block_slots_without_an_expert_add_nothing(sparse, weight, bad):
    """The result is that of weights of 0 on any expert, to the bit: a product of 0 adds nothing to
    a sum that starts at 0.  The workspace holds NaN everywhere beforehand."""
    x, routing, w, (gu, dn) = _block(sparse, torch.bfloat16)
    empty = torch.zeros_like(routing, dtype=torch.bool)
    empty[0, 1] = empty[7, 0] = empty[8, 2] = True
    empty[5] = empty[39] = True
    want = sp.moe_block(x, routing, w.masked_fill(empty, 0.0), gu, dn, 4, 512, 512)
    assert sp.last_device_error() == sp.OK
    ws = torch.full((sp.moe_block_workspace_bytes(40, 3, 4, 512, 512),), 255, dtype=torch.uint8, device="cuda")
    got = sp.moe_block(x, routing.masked_fill(empty, bad), w.masked_fill(empty, weight), gu, dn, 4, 512, 512, workspace=ws)
    torch.cuda.synchronize()
    sp.last_device_error()
    assert torch.isfinite(got).all() and torch.equal(got, want)
    assert not got[5].any() and not got[39].any()
