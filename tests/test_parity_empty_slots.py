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


def test_block_takes_what_the_router_gives():
    """moe_route on a padded batch (masked tokens, and tokens with fewer live experts than slots) into
    the block: no error, and the sum over the slots that have an expert."""
    x, _, _, (gu, dn) = _block(False, torch.bfloat16)
    logits = torch.randn(40, 4, generator=torch.Generator().manual_seed(2))
    logits[36:] = -float("inf")
    logits[3, :3] = -float("inf")
    logits[4, 1:] = float("nan")
    routing, w = sp.moe_route(logits.cuda(), 3)
    empty = routing < 0
    assert empty.sum() == 4 * 3 + 2 + 2
    y = sp.moe_block(x, routing, w, gu, dn, 4, 512, 512)
    torch.cuda.synchronize()
    assert sp.last_device_error() == sp.OK
    assert torch.equal(y, sp.moe_block(x, routing.masked_fill(empty, 0), w.masked_fill(empty, 0.0), gu, dn, 4, 512, 512))
    assert not y[36:].any()
    # a batch without any expert at all
    none = sp.moe_block(x, torch.full_like(routing, -1), w, gu, dn, 4, 512, 512)
    torch.cuda.synchronize()
    assert sp.last_device_error() == sp.OK and not none.any()


@pytest.mark.parametrize("form", ["16 bits", "nvfp4", "nvfp4 2:4"])
def test_grouped_slots_without_an_expert_are_zero(form):
    """Every path of the grouped product: no error, zeros there, the other slots as without them."""
    g = torch.Generator().manual_seed(3)
    E, N, K, T, topk = 5, 128, 512, 150, 3
    x = torch.randn(T, K, generator=g).bfloat16().cuda()
    w = (torch.randn(E * N, K, generator=g) * 0.05).bfloat16().cuda()
    if form == "nvfp4":
        w = sp.quantize_nvfp4(w)
    elif form == "nvfp4 2:4":
        v, m = sp.prune_compress_24(w)
        w = sp.Sparse24(sp.quantize_nvfp4(v), m)
    routing = torch.randint(0, E, (T, topk), generator=g).int().cuda()
    empty = torch.zeros_like(routing, dtype=torch.bool)
    empty[140:] = True
    empty[2, 1] = True
    want = sp.gemm_grouped(x, routing, w, E, N, K)
    got = torch.full((T, topk, N), float("nan"), device="cuda")
    sp.gemm_grouped(x, routing.masked_fill(empty, -1), w, E, N, K, out=got)
    torch.cuda.synchronize()
    assert sp.last_device_error() == sp.OK
    assert not got[empty].any()
    # 16 bits: sums of K slices by atomics in any order, at most K + 8 additions, each off by at most two
    # half steps (tensor cores may truncate), in either of the two results
    if form == "16 bits":
        bound = x.double().abs() @ w.double().abs().view(E, N, K).amax(0).t()
        err = (got - want)[~empty].double().abs()
        assert (err <= 4 * (K + 8) * 2.0 ** -24 * bound[:, None].expand(T, topk, N)[~empty]).all()
    else:
        assert torch.equal(got[~empty], want[~empty])
    # and the sorted form: rows behind the last expert's have no expert either
    s = sp.moe_sort(x, routing.masked_fill(empty, -1), E)
    s.xs[int(s.offsets[-1]):] = float("nan")
    rows = sp.gemm_grouped(s.xs, s.row_expert[:, None].contiguous(), w, E, N, K)[:, 0]
    torch.cuda.synchronize()
    assert sp.last_device_error() == sp.OK
    assert torch.isfinite(rows).all() and not rows[int(s.offsets[-1]):].any()


@pytest.mark.parametrize("N,off", [(128, 0), (256, 1), (384, 2), (128, 4)])
def test_grouped_zeros_stay_in_their_rows(N, off):
    """The tensor-core path into a y that starts off 16 bytes: slots without an expert first, last, alone
    and side by side; nothing beside y is written."""
    E, K, T, topk = 3, 256, 333, 3
    g = torch.Generator().manual_seed(N)
    x = torch.randn(T, K, generator=g).bfloat16().cuda()
    w = sp.quantize_nvfp4((torch.randn(E * N, K, generator=g) * 0.05).bfloat16().cuda())
    routing = torch.randint(0, E, (T, topk), generator=g).int()
    empty = torch.rand(T, topk, generator=g) < 0.2
    empty[0, 0] = empty[-1, -1] = True
    empty[50:80] = True
    routing, empty = routing.cuda(), empty.cuda()
    flat = torch.full((T * topk * N + off + 8,), 7.0, device="cuda")
    y = flat[off:off + T * topk * N].view(T, topk, N)
    sp.gemm_grouped(x, routing.masked_fill(empty, -1), w, E, N, K, out=y)
    torch.cuda.synchronize()
    assert sp.last_device_error() == sp.OK
    want = sp.gemm_grouped(x, routing, w, E, N, K).masked_fill(empty[..., None], 0.0)
    assert torch.equal(y, want)
    assert (flat[:off] == 7.0).all() and (flat[off + T * topk * N:] == 7.0).all()
