"""Edges of the 4-bit products: waits that run out in every form, experts over no entries, offsets that no sort
gives, several threads, and the way for many rows."""
import contextlib
import ctypes

import pytest
import torch

import fp16_gemm_b200 as sp
from test_parity_w4 import HALF, U, _cuda_ok, _gen, plain_values, random_w4


@contextlib.contextmanager
def _wait_limit(ns):
    old = ctypes.c_ulonglong()
    assert sp.lib().sp24_get_wait_limit(ctypes.byref(old)) == sp.OK
    assert sp.lib().sp24_set_wait_limit(ns) == sp.OK
    try:
        yield
    finally:
        assert sp.lib().sp24_set_wait_limit(old.value) == sp.OK


@pytest.mark.gpu
@pytest.mark.parametrize("act", [sp.ACT_NONE, sp.ACT_SWIGLU], ids=["none", "swiglu"])
@pytest.mark.parametrize("form", ["many items", "shared K", "x outside", "experts", "experts, shared K"])
def test_waits_that_run_out(form, act):
    """With a wait limit that most waits outlast, a call ends, and its result is right or it is
    reported; the next call is right."""
    dtype = torch.bfloat16
    M, N, K, E = {"many items": (2, 20000, 4096, 0), "shared K": (12, 48, 11232, 0), "x outside": (16, 9000, 9088, 0),
                  "experts": (70, 1024, 2048, 40), "experts, shared K": (5, 32, 9088, 3)}[form]
    x = torch.randn(M, K, generator=_gen(1)).to(dtype).cuda()
    w = random_w4(max(E, 1) * N, K, 32, True, dtype, 2)
    if E:
        counts = torch.randint(0, E, (M,), generator=_gen(3)).bincount(minlength=E)
        offsets = torch.cat((torch.zeros(1, dtype=torch.int64), counts.cumsum(0))).int().cuda()
        call = lambda: sp.gemv_w4_grouped(x, w, offsets, act)  # noqa: E731
    else:
        call = lambda: sp.gemv_w4(x, w, act)  # noqa: E731
    want = call()
    _cuda_ok()
    for limit in (1, 200, 1000, 3000):
        with _wait_limit(limit):
            y = call()
            status = sp.last_device_error()
        assert status == sp.ERR_DEVICE_TIMEOUT or (status == sp.OK and torch.equal(y, want))
    assert torch.equal(call(), want)
    _cuda_ok()


@pytest.mark.gpu
@pytest.mark.parametrize("act", [sp.ACT_NONE, sp.ACT_SWIGLU], ids=["none", "swiglu"])
@pytest.mark.parametrize("N", [2, 34, 3000])
@pytest.mark.parametrize("at", [[1, 4, 4, 6], [0, 30, 60, 61], [0, 0, 0, 0], [-3, 2, 70, 99]])
def test_experts_over_no_entries_write_only_their_rows(at, N, act):
    """K = 0: zeros in the rows that an expert has, the others as they were."""
    R, E = 64, 3
    none = sp.W4Tensor(torch.empty(E * N, 0, dtype=torch.uint8, device="cuda"),
                       torch.empty(E * N, 0, dtype=torch.bfloat16, device="cuda"))
    out = torch.full((R, N // 2 if act else N), -5.0, device="cuda")
    sp.gemv_w4_grouped(torch.empty(R, 0, dtype=torch.bfloat16, device="cuda"), none,
                       torch.tensor(at, dtype=torch.int32, device="cuda"), act, out=out)
    _cuda_ok()
    want = torch.full_like(out, -5.0)
    want[max(at[0], 0):min(at[-1], R)] = 0.0
    assert torch.equal(out, want)


@pytest.mark.gpu
@pytest.mark.parametrize("E,R", [(64, 100), (64, 3), (7000, 300), (4096, 1 << 25), (1 << 20, 65600)])
def test_offsets_that_name_rows_again_and_again(E, R):
    """Every other expert holds all rows: more tiles than any sorted rows have, in the larger cases more
    than 32 bits count.  The call ends soon, reports it and writes nothing beside y."""
    K = N = 32
    if R * E > 1 << 30:
        N = 1
    w = random_w4(64, K, 32, False, torch.float16, 1)
    w = sp.W4Tensor(w.codes[:N].repeat(E, 1), w.scales[:N].repeat(E, 1))
    x = torch.zeros(R, K, dtype=torch.float16, device="cuda")
    around = torch.full((R + 2, N), -5.0, device="cuda")
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1::2] = R
    sp.gemv_w4_grouped(x, w, offsets, out=around[1:-1])
    torch.cuda.synchronize()
    assert sp.last_device_error() == sp.ERR_INVALID_ARG
    assert (around[0] == -5).all() and (around[-1] == -5).all()
    # every row is the first expert's too, and every expert here is the same
    assert not around[1:-1].any()
    # the last expert alone has them: nothing is reported, and all are there
    offsets.zero_()
    offsets[-1] = R
    around[1:-1] = -5.0
    sp.gemv_w4_grouped(x, w, offsets, out=around[1:-1])
    _cuda_ok()
    assert not around[1:-1].any() and (around[0] == -5).all() and (around[-1] == -5).all()


@pytest.mark.gpu
def test_calls_of_several_threads():
    """First calls of a form from four host threads at once, each on a stream of its own."""
    import threading
    x = torch.randn(3, 1152, generator=_gen(1)).half().cuda()
    w = random_w4(70, 1152, 64, True, torch.float16, 2)
    torch.cuda.synchronize()
    got, start = [None] * 4, threading.Barrier(4)

    def work(i):
        stream = torch.cuda.Stream()
        start.wait()
        got[i] = [sp.gemv_w4(x, w, act, stream=stream) for act in (sp.ACT_NONE, sp.ACT_SWIGLU) for _ in range(8)]
        stream.synchronize()

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    _cuda_ok()
    want = [sp.gemv_w4(x, w, act) for act in (sp.ACT_NONE, sp.ACT_SWIGLU) for _ in range(8)]
    assert all(torch.equal(a, b) for r in got for a, b in zip(r, want))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
def test_many_rows_by_decoding_first(dtype):
    """The documented way for a prompt: decoded weights through the GEMM entry points, one matrix and
    experts with empty slots.  Each weight is off by half a step of its type; K products are added with
    at most K + 8 additions, each off by at most two half steps of fp32."""
    M, N, K, E = 150, 96, 256, 6
    x = torch.randn(M, K, generator=_gen(1)).to(dtype).cuda()
    w = random_w4(E * N, K, 64, True, dtype, 2)
    v, xd = plain_values(w).reshape(E, N, K), x.double().cpu()
    rel = HALF[dtype] + 2 * (K + 8) * U
    y = sp.gemm_dense(x, sp.dequantize_w4(sp.W4Tensor(*(t[:N] for t in w)), dtype))
    assert ((y.double().cpu() - xd @ v[0].t()).abs() <= rel * (xd.abs() @ v[0].abs().t())).all()
    ids = torch.randint(-1, E, (M, 2), generator=_gen(3)).int()
    s = sp.moe_sort(x, ids.cuda(), E)
    rows = sp.gemm_grouped(s.xs, s.row_expert[:, None].contiguous(), sp.dequantize_w4(w, dtype), E, N, K)[:, 0]
    got = sp.moe_unsort(rows.contiguous(), s.pos)
    _cuda_ok()
    held = (ids >= 0).double()[..., None]
    at = ids.clamp(min=0).long()
    want = (torch.einsum("tsnk,tk->tsn", v[at], xd) * held).sum(1)
    mag = (torch.einsum("tsnk,tk->tsn", v[at].abs(), xd.abs()) * held).sum(1)
    assert ((got.double().cpu() - want).abs() <= (rel + 2 * U) * mag).all()
