"""GPU parity of the 4-bit group weights: quantiser and dequantiser bit for bit against a plain
implementation of the definition, products against 64 bits.

Tolerances, u = 2^-24.  A product x (q - z) is exact in fp32 (8 or 11 bits times 5).  A group of G of
them is summed with at most G additions, each off by at most 2u of the sum of magnitudes (tensor
cores may truncate), scaled once (u), and the K / G groups and up to 16 partial sums are added
(u each): (2 G + K / G + 18) u on S = sum |x| |w|.  A 16-bit output adds half a step of its type.
SwiGLU: |SiLU'| <= 1.1 and expf is within 2 ulp, the quotient within 1: with the errors eg, eu of
gate and up, 1.1 eg |u| + (|SiLU(g)| + 1.1 eg) eu + 8u |h|.
"""
import numpy as np
import pytest
import torch

import fp16_gemm_b200 as sp

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -140, torch.bfloat16: 2.0 ** -125, torch.float16: 2.0 ** -25}
HALVES = [torch.bfloat16, torch.float16]


def _cuda_ok():
    torch.cuda.synchronize()
    assert sp.last_device_error() == sp.OK


def _gen(seed):
    return torch.Generator().manual_seed(seed)


# ------------------------------------------------------------------------------------ quantiser

def plain_quantize(w, G, with_zeros):
    """(q, scale in w's type, z) from the definition; the quotient of two 16-bit numbers in 64 bits."""
    R, K = w.shape
    v = w.double().cpu().reshape(R, K // G, G)
    lo, hi = v.amin(2).clamp(max=0), v.amax(2).clamp(min=0)
    if with_zeros:
        s = ((hi.float() - lo.float()) / torch.tensor(15.0)).to(w.dtype)
    else:
        s = (torch.maximum(hi, -lo).float() / torch.tensor(7.0)).to(w.dtype)
    s = torch.where(s.double() < 2.0 ** -126, torch.zeros_like(s), s)
    d = s.double()
    one = torch.where(d > 0, d, torch.ones_like(d))
    z = torch.full_like(d, 8.0)
    if with_zeros:
        z = torch.where(d > 0, torch.floor(-lo / one + 0.5).clamp(0, 15), torch.zeros_like(d))
    q = (torch.floor(v / one[..., None] + 0.5) + z[..., None]).clamp(0, 15)
    q = torch.where(d[..., None] > 0, q, z[..., None].expand_as(q))
    return q.reshape(R, K).to(torch.uint8), s, z.to(torch.uint8)


def codes_of(q):
    return q[:, 0::2] | (q[:, 1::2] << 4)


def plain_values(w):
    """float64 values of a W4Tensor on the CPU."""
    c = w.codes.cpu()
    q = torch.stack((c & 15, c >> 4), -1).reshape(c.shape[0], -1).double()
    G = q.shape[1] // w.scales.shape[1]
    s = w.scales.double().cpu().repeat_interleave(G, 1)
    z = 8.0 if w.zeros is None else (w.zeros.cpu() & 15).double().repeat_interleave(G, 1)
    return (q - z) * s


def _same_float(a, b):
    """Bitwise equal but for the sign of zero."""
    return torch.equal(a.cpu().float(), b.cpu().float())


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", HALVES, ids=["bf16", "f16"])
@pytest.mark.parametrize("R,K,G", [(1, 32, 32), (1, 128, 128), (3, 64, 64), (17, 160, 32), (5, 448, 64), (33, 896, 128),
                                   (257, 2080, 32), (1000, 1024, 128)])
def test_quantize(zeros, dtype, R, K, G):
    w = (torch.randn(R, K, generator=_gen(R + K)) * 0.02).to(dtype).cuda()
    got = sp.quantize_w4(w, G, zeros)
    q, s, z = plain_quantize(w, G, zeros)
    _cuda_ok()
    assert torch.equal(got.scales.cpu(), s)
    assert (got.zeros is None) == (not zeros) and (not zeros or torch.equal(got.zeros.cpu(), z))
    assert torch.equal(got.codes.cpu(), codes_of(q))
    for out in (torch.float32, torch.bfloat16, torch.float16):
        assert _same_float(sp.dequantize_w4(got, out), plain_values(got).to(out))


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", HALVES, ids=["bf16", "f16"])
def test_quantize_borders_and_extremes(zeros, dtype):
    """Quotients exactly on and one place beside every border, constant, one-sided, zero and
    subnormal groups, and groups at the type's extremes."""
    G, rows = 32, []
    f = torch.finfo(dtype)
    for s in (1.0, 0.75, 1.3359375, 2.0 ** -10, 0.0078125 * 1.5):
        top = [7 * s, -7 * s] if not zeros else [7.5 * s, -7.5 * s]
        border = torch.tensor([(n + 0.5) * s for n in range(-8, 8)], dtype=torch.float64).to(dtype)
        for x in (border, torch.nextafter(border, torch.full_like(border, 99.0)), torch.nextafter(border, torch.full_like(border, -99.0))):
            g = torch.zeros(G, dtype=dtype)
            g[:16] = x.clamp(-7 * s, 7 * s)
            g[16:18] = torch.tensor(top, dtype=torch.float64).to(dtype)
            rows.append(g)
    for g in (torch.zeros(G), -torch.zeros(G), torch.full((G,), 0.3), torch.full((G,), -0.3), torch.arange(G) * 0.1 + 1,
              -(torch.arange(G) * 0.1 + 1), torch.full((G,), f.max), torch.linspace(-1, 1, G) * f.max / 4,
              torch.full((G,), f.tiny), torch.linspace(-1, 1, G) * f.tiny, torch.full((G,), f.smallest_normal * f.eps),
              torch.cat((torch.tensor([f.max / 4]), torch.full((G - 1,), f.tiny)))):
        rows.append(g.to(dtype))
    w = torch.stack(rows).cuda()
    got = sp.quantize_w4(w, G, zeros)
    q, s, z = plain_quantize(w, G, zeros)
    _cuda_ok()
    assert torch.equal(got.scales.cpu(), s)
    assert not zeros or torch.equal(got.zeros.cpu(), z)
    assert torch.equal(got.codes.cpu(), codes_of(q))


def test_quantize_every_16_bit_quotient():
    """Every bf16 value of four binades against scales that take every significand."""
    G = 32
    v = torch.arange(0x3D80, 0x4000, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)  # 640 values, 1/16 .. 2
    tops = torch.arange(0x3F80, 0x4080, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)  # 256 maxima, 1 .. 4
    w = torch.zeros(len(tops), len(v) // 16, G, dtype=torch.bfloat16)
    w[:, :, :16] = v.reshape(1, -1, 16)
    w[:, :, 16:31] = -v.reshape(1, -1, 16)[..., :15]
    w[:, :, 31] = tops[:, None]
    w = w.reshape(len(tops), -1).cuda()
    for zeros in (False, True):
        got = sp.quantize_w4(w, G, zeros)
        q, s, z = plain_quantize(w, G, zeros)
        assert torch.equal(got.scales.cpu(), s) and torch.equal(got.codes.cpu(), codes_of(q))
        assert not zeros or torch.equal(got.zeros.cpu(), z)
    _cuda_ok()


def test_quantize_rows_do_not_leak():
    """A NaN or an infinity stays in its group."""
    w = (torch.randn(4, 256, generator=_gen(1)) * 0.02).bfloat16().cuda()
    clean = sp.quantize_w4(w, 64)
    w[1, 70], w[2, 5] = float("nan"), float("inf")
    got = sp.quantize_w4(w, 64)
    keep = torch.ones(4, 4, dtype=torch.bool)
    keep[1, 1] = keep[2, 0] = False
    assert torch.equal(got.codes.cpu().reshape(4, 4, 32)[keep], clean.codes.cpu().reshape(4, 4, 32)[keep])
    assert torch.equal(got.scales.cpu()[keep], clean.scales.cpu()[keep])


# ------------------------------------------------------------------------------------ products

def random_w4(rows, K, G, zeros, dtype, seed):
    g = _gen(seed)
    codes = torch.randint(0, 256, (rows, K // 2), generator=g).to(torch.uint8).cuda()
    scales = (torch.randn(rows, K // G, generator=g) * 0.01).to(dtype).cuda()
    z = torch.randint(0, 256, (rows, K // G), generator=g).to(torch.uint8).cuda() if zeros else None  # high bits are ignored
    return sp.W4Tensor(codes, scales, z)


def product_ref(x, w, rows=slice(None)):
    """(sums, tolerance) in 64 bits."""
    G = 2 * w.codes.shape[1] // w.scales.shape[1]
    part = sp.W4Tensor(w.codes[rows], w.scales[rows], None if w.zeros is None else w.zeros[rows])
    v, xd = plain_values(part), x.double().cpu()
    K = v.shape[1]
    return xd @ v.t(), (2 * G + K // G + 18) * U * (xd.abs() @ v.abs().t())


def swiglu_ref(v, tol):
    g, u = v.chunk(2, -1)
    eg, eu = tol.chunk(2, -1)
    silu = g / (1 + torch.exp(-g))
    h = silu * u
    return h, 1.1 * eg * u.abs() + (silu.abs() + 1.1 * eg) * eu + 8 * U * h.abs()


def assert_close(y, ref, tol):
    tol = tol + HALF[y.dtype] * (ref.abs() + tol) + TINY[y.dtype]
    bad = (y.double().cpu() - ref).abs() > tol
    assert not bad.any(), (bad.sum(), bad.nonzero()[:4], y.cpu()[bad][:4], ref[bad][:4], tol[bad][:4])


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype", HALVES, ids=["bf16", "f16"])
@pytest.mark.parametrize("M,N,K,G", [(1, 1, 32, 32), (1, 16, 128, 128), (2, 17, 96, 32), (3, 33, 192, 64), (7, 100, 384, 128),
                                     (8, 128, 1024, 32), (9, 65, 1056, 32), (16, 255, 640, 128), (33, 40, 448, 64),
                                     (5, 513, 2176, 128), (1, 1000, 4160, 32), (8, 300, 8192, 64), (70, 31, 256, 128)])
def test_gemv(zeros, dtype, M, N, K, G):
    x = torch.randn(M, K, generator=_gen(M + K)).to(dtype).cuda()
    w = random_w4(N, K, G, zeros, dtype, N)
    ref, tol = product_ref(x, w)
    y = sp.gemv_w4(x, w)
    y16 = sp.gemv_w4(x, w, dtype=dtype)
    _cuda_ok()
    assert y.dtype == torch.float32 and y16.dtype == dtype
    assert_close(y, ref, tol)
    assert_close(y16, ref, tol)
    assert torch.equal(y, sp.gemv_w4(x, w))  # the same bits again


@pytest.mark.parametrize("M,F,K,G", [(1, 1, 32, 32), (3, 15, 128, 64), (8, 17, 512, 128), (9, 100, 2048, 128), (16, 33, 96, 32)])
@pytest.mark.parametrize("dtype", HALVES, ids=["bf16", "f16"])
def test_gemv_swiglu(M, F, K, G, dtype):
    x = torch.randn(M, K, generator=_gen(M + K)).to(dtype).cuda()
    w = random_w4(2 * F, K, G, F % 2 == 1, dtype, F)
    ref, tol = swiglu_ref(*product_ref(x, w))
    y = sp.gemv_w4(x, w, sp.ACT_SWIGLU)
    assert y.dtype == dtype and y.shape == (M, F)
    assert_close(y, ref, tol)
    assert_close(sp.gemv_w4(x, w, sp.ACT_SWIGLU, dtype=torch.float32), ref, tol)
    _cuda_ok()


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("M,N,K", [(1, 70, 256), (3, 129, 384), (8, 33, 512), (11, 65, 512), (2, 47, 640), (8, 50, 16512),
                                   (16, 37, 9088), (20, 48, 1152), (1, 2400, 1920), (12, 48, 5248), (1, 2368, 3968), (1, 7000, 2560),
                                   (4, 4800, 1152)])
def test_gemv_paths(M, N, K, G, zeros):
    """One or two chunks of K, an x that does not fit shared memory, two tiles of rows, odd numbers of
    groups (rows of scales and zero points at every place within sixteen bytes)."""
    x = torch.randn(M, K, generator=_gen(M + K)).half().cuda()
    w = random_w4(N, K, G, zeros, torch.float16, N)
    y = sp.gemv_w4(x, w)
    assert_close(y, *product_ref(x, w))
    if N % 2 == 0:
        assert_close(sp.gemv_w4(x, w, sp.ACT_SWIGLU), *swiglu_ref(*product_ref(x, w)))
    _cuda_ok()


def test_gemv_waits_that_run_out():
    """With a wait limit that any wait outlasts, the call still ends, reports it at most, and the next
    one is right."""
    import ctypes
    x = torch.randn(2, 4096, generator=_gen(1)).bfloat16().cuda()
    w = random_w4(20000, 4096, 64, True, torch.bfloat16, 2)
    want = sp.gemv_w4(x, w)
    old = ctypes.c_ulonglong()
    assert sp.lib().sp24_get_wait_limit(ctypes.byref(old)) == sp.OK
    assert sp.lib().sp24_set_wait_limit(1) == sp.OK
    try:
        sp.gemv_w4(x, w)
        assert sp.last_device_error() in (sp.OK, sp.ERR_DEVICE_TIMEOUT)
    finally:
        assert sp.lib().sp24_set_wait_limit(old.value) == sp.OK
    assert torch.equal(sp.gemv_w4(x, w), want)
    _cuda_ok()


def test_gemv_two_streams_at_once():
    """Calls that overlap share nothing: the bits are those of calls made alone."""
    x = torch.randn(4, 2048, generator=_gen(1)).bfloat16().cuda()
    ws = [random_w4(3000, 2048, 64, True, torch.bfloat16, s) for s in range(2)]
    want = [sp.gemv_w4(x, w) for w in ws]
    streams = [torch.cuda.Stream() for _ in ws]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (w, st) in enumerate(zip(ws, streams)):
            got[i].append(sp.gemv_w4(x, w, stream=st))
    _cuda_ok()
    assert all(torch.equal(y, want[i]) for i in range(2) for y in got[i])


def test_gemv_scales_of_the_other_type():
    x = torch.randn(4, 256, generator=_gen(0)).bfloat16().cuda()
    w = random_w4(50, 256, 64, True, torch.float16, 1)
    assert_close(sp.gemv_w4(x, w), *product_ref(x, w))


def test_gemv_swiglu_far_ends():
    """Gates of +-1e4: SiLU is the gate itself, or 0, without a NaN."""
    K = 32
    codes = torch.full((4, K // 2), 0x99, dtype=torch.uint8).cuda()  # q - 8 = 1
    w = sp.W4Tensor(codes, torch.tensor([[300.0], [-300.0], [1.0], [1.0]]).half().cuda())
    y = sp.gemv_w4(torch.ones(1, K, device="cuda").half(), w, sp.ACT_SWIGLU, dtype=torch.float32)
    assert y[0, 0] == 9600 * 32 and y[0, 1] == 0


def test_gemv_non_finite_stays_in_its_row():
    x = torch.randn(3, 256, generator=_gen(2)).bfloat16().cuda()
    w = random_w4(40, 256, 64, False, torch.bfloat16, 3)
    clean = sp.gemv_w4(x, w)
    x[1, 17] = float("inf")
    w.scales[5, 2] = float("nan")
    y = sp.gemv_w4(x, w)
    rows = torch.ones(40, dtype=torch.bool)
    rows[5] = False
    assert torch.equal(y[0, rows], clean[0, rows]) and torch.equal(y[2, rows], clean[2, rows])
    assert torch.isnan(y[:, 5]).all() and not torch.isfinite(y[1]).any()


def test_gemv_writes_only_its_rows():
    x = torch.randn(5, 128, generator=_gen(4)).half().cuda()
    w = random_w4(33, 128, 128, False, torch.float16, 5)
    big = torch.full((7, 33), -9.0, device="cuda")
    sp.gemv_w4(x, w, out=big[1:6])
    assert (big[0] == -9).all() and (big[6] == -9).all() and torch.equal(big[1:6], sp.gemv_w4(x, w))
    assert sp.gemv_w4(x[:0], w).shape == (0, 33)
    assert sp.gemv_w4(x, sp.W4Tensor(w.codes[:0], w.scales[:0])).shape == (5, 0)
    none = sp.W4Tensor(w.codes[:, :0], w.scales[:, :0])
    assert (sp.gemv_w4(x[:, :0].contiguous(), none) == 0).all()
    _cuda_ok()


def test_gemv_codes_beyond_32_bits():
    """A matrix of more than 2^31 code bytes: rows at its end."""
    N, K = (1 << 20) + 24, 4160
    w = sp.W4Tensor(torch.zeros(N, K // 2, dtype=torch.uint8, device="cuda"),
                    torch.ones(N, K // 32, dtype=torch.bfloat16, device="cuda"))
    tail = random_w4(64, K, 32, False, torch.bfloat16, 8)
    w.codes[-64:], w.scales[-64:] = tail.codes, tail.scales
    x = torch.randn(2, K, generator=_gen(6)).bfloat16().cuda()
    y = sp.gemv_w4(x, w)
    _cuda_ok()
    assert_close(y[:, -64:], *product_ref(x, tail))
    first = x.double().cpu().sum(1) * -8
    assert ((y[:, 0].double().cpu() - first).abs() <= 4000 * U * 8 * x.double().cpu().abs().sum(1)).all()


# ------------------------------------------------------------------------------------ experts

def _grouped_ref(x, w, offsets, E, act):
    N = w.codes.shape[0] // E
    v = torch.zeros(x.shape[0], N, dtype=torch.float64)
    tol = torch.zeros_like(v)
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a < b:
            v[a:b], tol[a:b] = product_ref(x[a:b], w, slice(e * N, (e + 1) * N))
    return swiglu_ref(v, tol) if act == sp.ACT_SWIGLU else (v, tol)


@pytest.mark.parametrize("act", [sp.ACT_NONE, sp.ACT_SWIGLU], ids=["none", "swiglu"])
@pytest.mark.parametrize("counts,N,K,G,zeros,dtype", [
    ([1], 2, 32, 32, False, torch.bfloat16), ([0, 3, 0, 1, 8, 0], 48, 128, 64, True, torch.float16),
    ([9, 17, 1, 0, 40], 34, 256, 128, False, torch.bfloat16), ([0, 0, 0, 5], 130, 1056, 32, True, torch.bfloat16),
    ([2] * 70, 32, 96, 32, False, torch.float16), ([3, 0, 1, 9], 70, 512, 128, True, torch.bfloat16),
    ([1] * 40, 66, 2048, 64, False, torch.float16), ([30, 50], 48, 1184, 32, True, torch.bfloat16), ([0] * 300 + [1, 0, 16] + [0] * 50, 20, 512, 128, True, torch.bfloat16),
    ([0, 0, 1] * 900 + [0] * 4000 + [2, 9, 0, 0, 1] + [0] * 90, 2, 64, 64, False, torch.float16)])
def test_gemv_grouped(act, counts, N, K, G, zeros, dtype):
    E, live = len(counts), sum(counts)
    offsets = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32).cuda()
    R = live + 3  # three rows behind the last expert's
    x = torch.randn(R, K, generator=_gen(live)).to(dtype).cuda()
    x[live:] = float("nan")
    w = random_w4(E * N, K, G, zeros, dtype, N)
    cols = N // 2 if act else N
    out = torch.full((R, cols), -5.0, device="cuda")
    y = sp.gemv_w4_grouped(x, w, offsets, act, out=out)
    _cuda_ok()
    assert (y[live:] == -5).all()
    ref, tol = _grouped_ref(x, w, offsets, E, act)
    assert_close(y[:live], ref[:live], tol[:live])
    y16 = sp.gemv_w4_grouped(x, w, offsets, act, dtype=dtype)
    assert_close(y16[:live], ref[:live], tol[:live])
    assert (y16[live:] == 0).all()


def test_gemv_grouped_broken_offsets_stay_inside():
    """Offsets outside [0, R] are clamped and descending pairs hold nothing: rows elsewhere keep
    their values."""
    w = random_w4(4 * 16, 64, 32, False, torch.float16, 1)
    x = torch.randn(10, 64, generator=_gen(1)).half().cuda()
    out = torch.full((10, 16), -5.0, device="cuda")
    sp.gemv_w4_grouped(x, w, torch.tensor([-4, 2, 1, 8, 99], dtype=torch.int32).cuda(), out=out)
    _cuda_ok()
    for rows, e in ((slice(0, 2), 0), (slice(1, 8), 2), (slice(8, 10), 3)):
        ref, tol = product_ref(x[rows], w, slice(16 * e, 16 * e + 16))
        if e == 0:  # row 1 belongs to two experts here: row 0 to the first alone
            ref, tol, rows = ref[:1], tol[:1], slice(0, 1)
        if e == 2:
            ref, tol, rows = ref[1:], tol[1:], slice(2, 8)
        assert_close(out[rows], ref, tol)


def test_stream_device_and_graph():
    x = torch.randn(4, 512, generator=_gen(3)).bfloat16().cuda()
    w16 = (torch.randn(96, 512, generator=_gen(4)) * 0.02).bfloat16().cuda()

    def chain(stream=None):
        q = sp.quantize_w4(w16, 64, True, stream=stream)
        return [*q, sp.dequantize_w4(q, stream=stream), sp.gemv_w4(x, q, stream=stream),
                sp.gemv_w4(x, q, sp.ACT_SWIGLU, stream=stream)]

    want = chain()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = chain(side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = chain()
    x.copy_(torch.randn(4, 512, generator=_gen(5)))
    w16.copy_(torch.randn(96, 512, generator=_gen(6)))
    graph.replay()
    again = [t.clone() for t in held]
    assert all(torch.equal(a, b) for a, b in zip(again, chain()))
    _cuda_ok()


def test_refusals():
    x = torch.zeros(2, 128, dtype=torch.bfloat16, device="cuda")
    w = random_w4(8, 128, 64, False, torch.bfloat16, 0)
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    for call, err in ((lambda: sp.quantize_w4(x.float()), TypeError), (lambda: sp.quantize_w4(x, 48), ValueError),
                      (lambda: sp.quantize_w4(x[:, :96], 32), ValueError), (lambda: sp.gemv_w4(x.float(), w), TypeError),
                      (lambda: sp.gemv_w4(x[:, :64].contiguous(), w), ValueError), (lambda: sp.gemv_w4(x, w, 7), sp.SP24Error),
                      (lambda: sp.gemv_w4(x, w, dtype=torch.float16), TypeError),
                      (lambda: sp.gemv_w4(x, sp.W4Tensor(w.codes, w.scales[:, :1].contiguous().repeat(1, 3))), ValueError),
                      (lambda: sp.gemv_w4(x, sp.W4Tensor(w.codes[:, :16].contiguous(), w.scales)), ValueError),
                      (lambda: sp.gemv_w4(x, sp.W4Tensor(w.codes[:7], w.scales[:7]), sp.ACT_SWIGLU), sp.SP24Error),
                      (lambda: sp.gemv_w4_grouped(x, w, torch.zeros(4, dtype=torch.int32, device="cuda")), ValueError),
                      (lambda: sp.gemv_w4_grouped(x, w, off.long()), TypeError),
                      (lambda: sp.gemv_w4(x, w, out=torch.zeros(2, 9, device="cuda")), ValueError),
                      (lambda: sp.gemv_w4(x, sp.W4Tensor(w.codes.cpu(), w.scales)), ValueError)):
        with pytest.raises(err):
            call()


def test_refusals_of_given_outputs_and_types():
    w16 = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    plain, offset = sp.quantize_w4(w16, 64), sp.quantize_w4(w16, 64, True)
    for call, err in ((lambda: sp.quantize_w4(w16, 64, False, out=offset), ValueError),
                      (lambda: sp.quantize_w4(w16, 64, True, out=plain), ValueError),
                      (lambda: sp.dequantize_w4(plain, torch.int32), TypeError),
                      (lambda: sp.dequantize_w4(plain, torch.float64), TypeError),
                      (lambda: sp.dequantize_w4(plain, out=w16), TypeError)):
        with pytest.raises(err):
            call()
    _cuda_ok()


def test_graph_of_branches_behind_copies():
    """Captured launches that follow a fill or a copy, and ones that follow two joined branches."""
    x = torch.randn(4, 512, generator=_gen(3)).bfloat16().cuda()
    w16 = (torch.randn(96, 512, generator=_gen(4)) * 0.02).bfloat16().cuda()
    held, staged = torch.empty_like(x), torch.empty_like(w16)
    y, z = torch.empty(4, 96, device="cuda"), torch.empty(4, 96, device="cuda")
    side = torch.cuda.Stream()

    def chain():
        y.zero_()
        held.copy_(x)
        staged.copy_(w16)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            a = sp.quantize_w4(staged, 64, True)
            sp.gemv_w4(held, a, out=z)
        b = sp.quantize_w4(staged, 32)
        sp.gemv_w4(held, b, out=y)
        torch.cuda.current_stream().wait_stream(side)
        v, u = sp.dequantize_w4(a), sp.dequantize_w4(b)
        return [y.clone(), z.clone(), v, u, sp.gemv_w4(held, a)]

    chain()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain()
    for seed in range(5, 9):
        x.copy_(torch.randn(4, 512, generator=_gen(seed)))
        w16.copy_(torch.randn(96, 512, generator=_gen(seed + 9)) * 0.02)
        graph.replay()
        graph.replay()
        again = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(again, chain()))
        torch.cuda.synchronize()
    _cuda_ok()
