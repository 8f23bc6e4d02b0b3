"""The routed feed-forward's operators run together: a decode step with 4-bit experts, and a
training step whose gradients are checked against differences of the 64-bit definition."""
import numpy as np
import pytest
import torch

import fp16_gemm_b200 as sp
from test_parity_w4 import HALF, U, plain_values, random_w4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16], ids=["bf16", "f16"])
@pytest.mark.parametrize("T,E,k,H,F", [(1, 16, 4, 128, 64), (8, 32, 6, 256, 96), (40, 8, 2, 64, 160)])
def test_decode_step(dtype, T, E, k, H, F):
    """router logits -> route -> sort -> gate / up with SwiGLU -> down -> unsort."""
    g = torch.Generator().manual_seed(T + E)
    x = torch.randn(T, H, generator=g).to(dtype).cuda()
    logits = torch.randn(T, E, generator=g).cuda()
    if T > 2:
        logits[-1] = -float("inf")  # a padded token
    gu = random_w4(E * 2 * F, H, 32, False, dtype, 1)
    dn = random_w4(E * H, F, 32, True, dtype, 2)
    routing, w = sp.moe_route(logits, k)
    s = sp.moe_sort(x, routing, E)
    h = sp.gemv_w4_grouped(s.xs, gu, s.offsets, sp.ACT_SWIGLU)
    y = sp.gemv_w4_grouped(h, dn, s.offsets)
    out = sp.moe_unsort(y, s.pos, w, dtype=dtype)
    torch.cuda.synchronize()
    assert sp.last_device_error() == sp.OK
    # the definition in 64 bits, with h rounded to its type as the step's definition has it: h may
    # fall to the neighbouring step, so each |h| counts with a whole step of it (two halves)
    G, D = plain_values(gu).reshape(E, 2 * F, H), plain_values(dn).reshape(E, H, F)
    xd = x.double().cpu()
    ids, wd = routing.cpu().numpy(), w.double().cpu()
    want, tol = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            if e < 0:
                continue
            v, mag = G[e] @ xd[t], G[e].abs() @ xd[t].abs()
            a, b = v[:F], v[F:]
            hd = a / (1 + torch.exp(-a)) * b
            eh = 200 * U * (1.1 * mag[:F] * b.abs() + (a.abs() + 1) * mag[F:]) + 2 * HALF[dtype] * hd.abs()
            want[t] += wd[t, j] * (D[e] @ hd)
            tol[t] += wd[t, j].abs() * (D[e].abs() @ (eh + 200 * U * hd.abs()))
    tol += HALF[dtype] * (want.abs() + tol) + k * U * want.abs() + 1e-7
    assert ((out.double().cpu() - want).abs() <= tol).all()
    assert T <= 2 or (out[-1] == 0).all()


def test_decode_steps_without_a_wait_between():
    """The step repeated on new tokens with nothing waited for in between, weights quantised on the way."""
    T, E, k, H, F = 8, 32, 6, 256, 96
    g = torch.Generator().manual_seed(1)
    xs = [torch.randn(T, H, generator=g).bfloat16().cuda() for _ in range(3)]
    ls = [torch.randn(T, E, generator=g).cuda() for _ in range(3)]
    wg = (torch.randn(E * 2 * F, H, generator=g) * 0.05).bfloat16().cuda()
    wd = (torch.randn(E * H, F, generator=g) * 0.05).bfloat16().cuda()

    def step(x, l, done):
        gu, dn = sp.quantize_w4(wg, 64, True), sp.quantize_w4(wd, 32)
        done()
        routing, w = sp.moe_route(l, k)
        done()
        s = sp.moe_sort(x, routing, E)
        done()
        h = sp.gemv_w4_grouped(s.xs, gu, s.offsets, sp.ACT_SWIGLU)
        done()
        y = sp.gemv_w4_grouped(h, dn, s.offsets)
        done()
        return sp.moe_unsort(y, s.pos, w), sp.dequantize_w4(dn)

    want = [step(x, l, torch.cuda.synchronize) for x, l in zip(xs, ls)]
    got = [step(xs[i % 3], ls[i % 3], lambda: None) for i in range(18)]
    torch.cuda.synchronize()
    assert sp.last_device_error() == sp.OK
    assert all(torch.equal(a, b) for i, r in enumerate(got) for a, b in zip(r, want[i % 3]))


@pytest.mark.parametrize("form", [(sp.ROUTE_SOFTMAX, True), (sp.ROUTE_SOFTMAX, False), (sp.ROUTE_SIGMOID, True)],
                         ids=["softmax_renorm", "softmax", "sigmoid_renorm"])
def test_training_step(form):
    """L = sum r * unsort(f(sort(x)), w(logits)) with f a matrix per expert (the package's grouped
    product): the gradients of x and of the logits against central differences in 64 bits."""
    T, E, k, H = 12, 8, 3, 64
    rng = np.random.default_rng(3)
    logits = rng.standard_normal((T, E)).astype(np.float32)
    x = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32)).bfloat16()
    A = torch.from_numpy((rng.standard_normal((E, H, H)) / 8).astype(np.float32)).bfloat16()
    r = torch.from_numpy(rng.standard_normal((T, H)).astype(np.float32))

    routing, w = sp.moe_route(torch.from_numpy(logits).cuda(), k, *form)
    s = sp.moe_sort(x.cuda(), routing, E)
    # rows in expert order with their expert as the only slot: the routed product of the package
    ys = sp.gemm_grouped(s.xs, s.row_expert[:, None].contiguous(), A.reshape(E * H, H).contiguous().cuda(), E, H, H)[:, 0]
    y = sp.moe_unsort(ys.contiguous(), s.pos, w)
    dys, dw = sp.moe_unsort_backward(r.cuda(), ys.contiguous(), s.pos, w)
    dxs = torch.bmm(A.float().cuda().transpose(1, 2)[s.row_expert.long()], dys[..., None])[..., 0]
    dx = sp.moe_sort_backward(dxs.contiguous(), s.pos).double().cpu().numpy()
    dl = sp.moe_route_backward(dw, torch.from_numpy(logits).cuda(), routing, *form).double().cpu().numpy()
    torch.cuda.synchronize()
    assert sp.last_device_error() == sp.OK

    ids = routing.cpu().numpy()
    Ad, rd, xd = A.double().numpy(), r.double().numpy(), x.double().numpy()

    def weights(l):
        out = np.zeros((T, k))
        for t in range(T):
            v = l[t, ids[t]]
            if form[0] == sp.ROUTE_SOFTMAX:
                out[t] = np.exp(v) / (np.exp(v).sum() if form[1] else np.exp(l[t]).sum())
            else:
                q = 1 / (1 + np.exp(-v))
                out[t] = q / q.sum()
        return out

    def loss(l, xx):
        f = np.einsum("tkij,tj->tki", Ad[ids], xx)
        return (weights(l)[..., None] * f * rd[:, None]).sum()

    f = np.einsum("tkij,tj->tki", Ad[ids], xd)
    full = (weights(logits.astype(np.float64))[..., None] * f).sum(1)
    assert np.abs(y.double().cpu().numpy() - full).max() < 1e-4  # fp32 sums of 64 products of magnitude 1 / 8
    l64 = logits.astype(np.float64)
    for _ in range(60):
        t, e, h = int(rng.integers(T)), int(rng.integers(E)), int(rng.integers(H))
        step = np.zeros_like(l64)
        step[t, e] = 1e-4
        num = (loss(l64 + step, xd) - loss(l64 - step, xd)) / 2e-4
        # |dw| is at most sum |r f|, some hundreds here: fp32 keeps 2^-24 of that per term, 64 terms
        # (1e-3 at most), the differences 1e-8 of it
        assert abs(num - dl[t, e]) < 1e-3
        step = np.zeros_like(xd)
        step[t, h] = 1e-3
        num = (loss(l64, xd + step) - loss(l64, xd - step)) / 2e-3
        assert abs(num - dx[t, h]) < 1e-4  # linear in x
