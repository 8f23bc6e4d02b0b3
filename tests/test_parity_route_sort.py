"""GPU parity of the router, the token sort and the unsort, and their gradients, against plain
implementations in 64 bits on the CPU.

Tolerances, u = 2^-24 (fp32 half step), derived per output:
  exp(l - m) in fp32: the argument is off by |l - m| u, expf by 2 ulp = 4u, so a weight (one quotient,
  a sum of up to 1024 such terms in at most 32 + 5 additions) is off by at most
  (2 D + 8 + 37 + 2) u relative, D the largest |l - m| of the row's finite logits.
  A gradient is a short sum of products of weights and given numbers: the same relative error on
  the sum of its terms' magnitudes, twice (two weights meet in a product), plus half a step of the
  output's type.
  unsort: topk fp32 fmas, so topk u on the sum of magnitudes, plus half a step of the output's type;
  the dot products H u (any order of H additions).
"""
import numpy as np
import pytest
import torch

import fp16_gemm_b200 as sp

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -140, torch.bfloat16: 2.0 ** -125, torch.float16: 2.0 ** -25}
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def _cuda_ok():
    torch.cuda.synchronize()
    assert sp.last_device_error() == sp.OK


# ------------------------------------------------------------------------------------ router

def plain_route(l, k, scoring, renorm):
    """Routing, weights and the sum-of-magnitudes scale, from float64 logits [T, E] (numpy)."""
    T, E = l.shape
    ids = np.full((T, k), -1, np.int32)
    w = np.zeros((T, k))
    for t in range(T):
        order = [e for e in sorted(range(E), key=lambda e: (-l[t, e] if l[t, e] == l[t, e] else np.inf, e))
                 if l[t, e] == l[t, e] and l[t, e] > -np.inf][:k]
        if not order:
            continue
        ids[t, :len(order)] = order
        v = l[t, order]
        if scoring == sp.ROUTE_SOFTMAX:
            m = v[0]
            total = np.exp(v - m).sum() if renorm else np.exp(l[t] - m).sum()
            w[t, :len(order)] = np.exp(v - m) / total
        else:
            s = 1 / (1 + np.exp(-v))
            w[t, :len(order)] = s / s.sum() if renorm else s
    return ids, w


def plain_route_backward(l, ids, dw, scoring, renorm):
    """(gradient, sum of its terms' magnitudes)."""
    T, E = l.shape
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        slots = [s for s in range(ids.shape[1]) if ids[t, s] >= 0]
        if not slots:
            continue
        at, g = ids[t, slots], dw[t, slots]
        v = l[t, at]
        if scoring == sp.ROUTE_SOFTMAX:
            m = v.max() if renorm else l[t].max()
            w = np.exp(v - m) / (np.exp(v - m).sum() if renorm else np.exp(l[t] - m).sum())
            if renorm:
                np.add.at(d[t], at, w * (g - (w * g).sum()))
                np.add.at(mag[t], at, w * (np.abs(g) + (w * np.abs(g)).sum()))
            else:
                p = np.exp(l[t] - m) / np.exp(l[t] - m).sum()
                np.add.at(d[t], at, w * g)
                np.add.at(mag[t], at, w * np.abs(g))
                d[t] -= p * (w * g).sum()
                mag[t] += p * (w * np.abs(g)).sum()
        else:
            s = 1 / (1 + np.exp(-v))
            slope = s * (1 / (1 + np.exp(v)))
            if renorm:
                np.add.at(d[t], at, slope * (g - (s * g).sum() / s.sum()) / s.sum())
                np.add.at(mag[t], at, slope * (np.abs(g) + (s * np.abs(g)).sum() / s.sum()) / s.sum())
            else:
                np.add.at(d[t], at, slope * g)
                np.add.at(mag[t], at, slope * np.abs(g))
    return d, mag


def _spread(l):
    f = np.where(np.isfinite(l), l, 0.0)
    return float(np.abs(f).max() * 2) + 1


def _check_route(logits, k, scoring, renorm, seed=0):
    l = logits.double().cpu().numpy()
    routing, w = sp.moe_route(logits, k, scoring, renorm)
    _cuda_ok()
    with np.errstate(invalid="ignore"):
        ids, ref = plain_route(l, k, scoring, renorm)
    assert np.array_equal(routing.cpu().numpy(), ids)
    got = w.double().cpu().numpy()
    rel = (2 * _spread(l) + 47) * U
    assert (np.abs(got - ref) <= rel * np.abs(ref) + TINY[torch.float32]).all()
    g = torch.from_numpy(np.random.default_rng(seed).standard_normal(ids.shape).astype(np.float32)).cuda()
    g[routing < 0] = float("nan")  # what stands at an empty slot does not count
    d = sp.moe_route_backward(g, logits, routing, scoring, renorm)
    _cuda_ok()
    with np.errstate(invalid="ignore"):
        ref, mag = plain_route_backward(l, ids, g.double().cpu().numpy(), scoring, renorm)
    got = d.double().cpu().numpy()
    tol = 2 * rel * mag + HALF[logits.dtype] * np.abs(ref) + TINY[logits.dtype]
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4], tol[bad][:4])


FORMS = [(sp.ROUTE_SOFTMAX, True), (sp.ROUTE_SOFTMAX, False), (sp.ROUTE_SIGMOID, True), (sp.ROUTE_SIGMOID, False)]


@pytest.mark.parametrize("form", FORMS, ids=["softmax_renorm", "softmax", "sigmoid_renorm", "sigmoid"])
@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 5, 5), (5, 32, 8), (7, 33, 2), (4, 100, 32), (9, 160, 6),
                                   (6, 512, 10), (2, 777, 3), (3, 1024, 32), (130, 64, 4)])
def test_route(form, dtype, T, E, k):
    g = torch.Generator().manual_seed(T * 1000 + E)
    _check_route((torch.randn(T, E, generator=g) * 2).to(dtype).cuda(), k, *form)


@pytest.mark.parametrize("form", FORMS, ids=["softmax_renorm", "softmax", "sigmoid_renorm", "sigmoid"])
def test_route_ties_masks_and_signed_zeros(form):
    """Equal logits go to the lower expert (also across lanes and registers), +0 and -0 are equal,
    -inf is never selected, and a row of -inf selects nothing."""
    E, k = 96, 6
    l = torch.zeros(8, E)
    l[0, ::2] = -0.0
    l[1] = 1.0
    l[1, 40] = 2.0
    l[1, 71] = 2.0
    l[2] = -float("inf")
    l[3] = -float("inf")
    l[3, 90] = -3.0
    l[3, 7] = -3.0
    l[4] = torch.arange(E) % 3
    l[5] = -float("inf")
    l[5, E - 1] = 0.0
    l[6] = -60.0 + torch.arange(E) * 0.5
    l[7, 64:] = -float("inf")
    _check_route(l.cuda(), k, *form)


def test_route_nan_is_not_selected():
    l = torch.randn(3, 40, generator=torch.Generator().manual_seed(5))
    l[0, 3] = float("nan")
    l[1, :39] = float("nan")
    l[2] = float("nan")
    c = l.cuda()
    routing, w = sp.moe_route(c, 4, sp.ROUTE_SOFTMAX, True)
    ids, ref = plain_route(l.double().numpy(), 4, sp.ROUTE_SOFTMAX, True)
    assert np.array_equal(routing.cpu().numpy(), ids)
    assert np.allclose(w.cpu().numpy(), ref, rtol=100 * U, atol=0)
    _, w = sp.moe_route(c, 4, sp.ROUTE_SOFTMAX, False)  # the sum is over all experts: NaN shows
    assert torch.isnan(w[:1]).all() and torch.isnan(w[1, 0]) and (w[1, 1:] == 0).all() and (w[2] == 0).all()


def test_route_backward_repeated_and_bad_ids():
    """An id met twice collects both slots; an id out of range is an empty slot and is reported."""
    l = torch.randn(4, 48, generator=torch.Generator().manual_seed(6)).cuda()
    ids = torch.tensor([[3, 3, 3], [40, 7, 40], [-1, 5, -1], [9, -1, 9]], dtype=torch.int32).cuda()
    g = torch.randn(4, 3, generator=torch.Generator().manual_seed(7)).cuda()
    for form in FORMS:
        d = sp.moe_route_backward(g, l, ids, *form)
        _cuda_ok()
        ref, mag = plain_route_backward(l.double().cpu().numpy(), ids.cpu().numpy(), g.double().cpu().numpy(), *form)
        assert (np.abs(d.double().cpu().numpy() - ref) <= 2 * (2 * _spread(l.cpu().numpy()) + 47) * U * mag + TINY[torch.float32]).all()
        bad = ids.clone()
        bad[2, 0], bad[2, 2] = 48, -2
        assert torch.equal(sp.moe_route_backward(g, l, bad, *form), d)
        assert sp.last_device_error() == sp.ERR_INVALID_ARG


@pytest.mark.parametrize("form", FORMS, ids=["softmax_renorm", "softmax", "sigmoid_renorm", "sigmoid"])
def test_route_gradient_against_differences(form):
    """The gradient against central differences of the 64-bit definition (selection held)."""
    rng = np.random.default_rng(11)
    l = torch.from_numpy(rng.standard_normal((2, 24)).astype(np.float32))
    g = torch.from_numpy(rng.standard_normal((2, 5)).astype(np.float32))
    routing, _ = sp.moe_route(l.cuda(), 5, *form)
    d = sp.moe_route_backward(g.cuda(), l.cuda(), routing, *form).double().cpu().numpy()
    ids, ld = routing.cpu().numpy(), l.double().numpy()

    def loss(a):
        w = np.zeros((2, 5))
        for t in range(2):
            v = a[t, ids[t]]
            if form[0] == sp.ROUTE_SOFTMAX:
                w[t] = np.exp(v) / (np.exp(v).sum() if form[1] else np.exp(a[t]).sum())
            else:
                s = 1 / (1 + np.exp(-v))
                w[t] = s / s.sum() if form[1] else s
        return (w * g.double().numpy()).sum()

    for t in range(2):
        for e in range(24):
            step = np.zeros_like(ld)
            step[t, e] = 1e-4
            # central differences at 1e-4: third derivatives are below 10, so below 2e-8 off; the
            # kernel's fp32 terms are below 1 in magnitude: 100 u
            assert abs((loss(ld + step) - loss(ld - step)) / 2e-4 - d[t, e]) < 1e-7 + 100 * U


# ------------------------------------------------------------------------------------ sort

def plain_sort(routing, E):
    """The stable order, by Python's own sort."""
    T, k = routing.shape
    flat = routing.reshape(-1)
    held = [i for i in range(T * k) if 0 <= flat[i] < E]
    order = sorted(held, key=lambda i: flat[i])
    pos = np.full(T * k, -1, np.int32)
    src = np.full(T * k, -1, np.int32)
    row_expert = np.full(T * k, -1, np.int32)
    for r, i in enumerate(order):
        pos[i], src[r], row_expert[r] = r, i, flat[i]
    offsets = np.array([sum(1 for i in held if flat[i] < e) for e in range(E + 1)], np.int32) if T * k * E < 10**6 else \
        np.concatenate([[0], np.cumsum(np.bincount(flat[held], minlength=E))]).astype(np.int32)
    return pos.reshape(T, k), src, row_expert, offsets


def _check_sort(routing, E, H, dtype, seed=0):
    T, k = routing.shape
    n = T * k
    x = torch.randn(T, H, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()
    r = torch.from_numpy(routing).cuda()
    sentinel = torch.full((n, H), 7.0, dtype=dtype, device="cuda")
    i32 = lambda *s: torch.full(s, 77, dtype=torch.int32, device="cuda")  # noqa: E731
    got = sp.moe_sort(x, r, E, out=(sentinel, i32(T, k), i32(n), i32(n), i32(E + 1)))
    torch.cuda.synchronize()
    pos, src, row_expert, offsets = plain_sort(routing, E)
    for a, b in ((got.pos, pos), (got.src, src), (got.row_expert, row_expert), (got.offsets, offsets)):
        assert np.array_equal(a.cpu().numpy(), b)
    want = torch.full((n, H), 7.0, dtype=dtype)  # rows behind the last are left as they were
    live = offsets[-1]
    want[:live] = x.cpu()[torch.from_numpy(src[:live].astype(np.int64) // k)]
    assert torch.equal(got.xs.cpu(), want)
    tables = sp.moe_sort_tables(r, E)
    assert tables.xs is None and all(torch.equal(a, b) for a, b in zip(tables[1:], got[1:]))
    return x, r, got


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 1), (1, 2, 3, 8), (8, 10, 512, 64), (33, 3, 7, 129), (100, 4, 16, 2),
                                     (257, 2, 5, 40), (64, 8, 64, 1000), (300, 10, 40, 16), (1000, 7, 333, 24)])
def test_sort(dtype, T, k, E, H):
    rng = np.random.default_rng(T + E)
    _check_sort(rng.integers(0, E, (T, k)).astype(np.int32), E, H, dtype)
    sp.last_device_error()


@pytest.mark.parametrize("T,k,E", [(5000, 2, 9), (4096, 10, 512), (1024, 2, 7), (1025, 2, 7), (300, 2, 20000), (9000, 1, 30000), (3001, 5, 1030), (60000, 1, 3), (20011, 8, 128)])
def test_sort_many(T, k, E):
    """Many entries: skewed experts (some empty, one with a third of all), padded tokens."""
    rng = np.random.default_rng(E)
    r = (rng.random((T, k)) ** 3 * E).astype(np.int32)
    r[rng.random((T, k)) < 0.3] = E // 2
    r[T - T // 9:] = -1
    _check_sort(r, E, 8, torch.bfloat16)
    _cuda_ok()


def test_sort_one_expert_and_no_entry():
    _check_sort(np.full((700, 3), 2, np.int32), 4, 16, torch.bfloat16)  # everything on one expert
    x, r, got = _check_sort(np.full((50, 2), -1, np.int32), 4, 16, torch.bfloat16)  # nothing anywhere
    _cuda_ok()
    assert (got.offsets == 0).all()
    empty = sp.moe_sort(torch.zeros(0, 16, device="cuda"), torch.zeros(0, 2, dtype=torch.int32, device="cuda"), 5)
    _cuda_ok()
    assert empty.xs.shape == (0, 16) and (empty.offsets == 0).all() and empty.offsets.numel() == 6
    none = sp.moe_sort(torch.zeros(4, 0, device="cuda"), torch.zeros(4, 2, dtype=torch.int32, device="cuda"), 5)
    _cuda_ok()
    assert none.offsets.tolist() == [0, 8, 8, 8, 8, 8]


@pytest.mark.parametrize("T", [20, 3000])
def test_sort_reports_bad_ids(T):
    r = np.random.default_rng(2).integers(0, 6, (T, 2)).astype(np.int32)
    r[3, 1], r[T - 1, 0], r[7, 0] = 6, -2, 2**31 - 1
    _check_sort(r, 6, 8, torch.float32)
    assert sp.last_device_error() == sp.ERR_INVALID_ARG


def test_sort_unaligned_rows():
    """Row bases off 16 bytes (a view one row into an odd-width tensor)."""
    base = torch.randn(40, 13, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    x = base[1:]
    r = torch.from_numpy(np.random.default_rng(4).integers(0, 5, (39, 2)).astype(np.int32)).cuda()
    got = sp.moe_sort(x, r, 5)
    assert torch.equal(got.xs, x[(got.src // 2).long()])


# ------------------------------------------------------------------------------------ unsort

def _check_unsort(ys, pos, w, odt, seed=0):
    T, k = pos.shape
    rows, H = ys.shape
    p = pos.cpu().numpy()
    live = (p >= 0) & (p < rows)
    at = np.where(live, p, 0)
    y64 = ys.double().cpu().numpy()
    w64 = np.where(live, w.double().cpu().numpy() if w is not None else 1.0, 0.0)
    y = sp.moe_unsort(ys, pos, w, dtype=odt)
    terms = np.where(live[..., None], y64[at], 0.0) * w64[..., None]
    ref, mag = terms.sum(1), np.abs(terms).sum(1)
    tol = k * U * mag + HALF[odt] * (np.abs(ref) + k * U * mag) + TINY[odt]
    assert (np.abs(y.double().cpu().numpy() - ref) <= tol).all()
    dy = torch.randn(T, H, generator=torch.Generator().manual_seed(seed)).to(odt).cuda()
    outs = (torch.full_like(ys, 7.0), torch.full((T, k), 7.0, device="cuda"))
    dys, dw = sp.moe_unsort_backward(dy, ys, pos, w, out=outs)
    d64 = dy.double().cpu().numpy()
    want = np.full((rows, H), 7.0)
    prod = d64[:, None] * w64[..., None]
    want[p[live]] = prod[live]
    tol = (HALF[ys.dtype] + U) * np.abs(want) * 1.01 + TINY[ys.dtype]
    assert (np.abs(dys.double().cpu().numpy() - want) <= tol).all()
    dots = d64[:, None] * np.where(live[..., None], y64[at], 0.0)
    assert (np.abs(dw.double().cpu().numpy() - dots.sum(2)) <= (H + 1) * U * np.abs(dots).sum(2) + TINY[torch.float32]).all()
    assert (dw.cpu().numpy()[~live] == 0).all()
    return y, dys, dw


PAIRS = [(torch.float32, torch.float32), (torch.float32, torch.bfloat16), (torch.float32, torch.float16),
         (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32), (torch.float16, torch.float16),
         (torch.float16, torch.float32)]


@pytest.mark.parametrize("pair", PAIRS, ids=lambda p: "-".join(str(d)[6:] for d in p))
@pytest.mark.parametrize("T,k,H", [(1, 1, 1), (2, 3, 7), (8, 10, 2048), (17, 2, 130), (5, 33, 36), (3, 64, 8), (70, 4, 264),
                                   (6, 5, 1004)])
def test_unsort(pair, T, k, H):
    rng = np.random.default_rng(T * 100 + H)
    g = torch.Generator().manual_seed(H)
    r = rng.integers(0, 12, (T, k)).astype(np.int32)
    if T > 2:
        r[T - 1] = -1  # a padded token: its y is 0
        r[0, 0] = -1
    pos = sp.moe_sort_tables(torch.from_numpy(r).cuda(), 12).pos
    ys = torch.randn(T * k, H, generator=g).to(pair[0]).cuda()
    w = torch.rand(T, k, generator=g).cuda()
    if T > 2:
        w[0, 0] = float("nan")  # at an empty slot
    y, _, _ = _check_unsort(ys, pos, w, pair[1])
    _cuda_ok()
    assert T <= 2 or (y[T - 1] == 0).all()


def test_unsort_without_weights_is_the_sorts_gradient():
    rng = np.random.default_rng(1)
    x, r, got = _check_sort(rng.integers(-1, 9, (60, 4)).astype(np.int32), 9, 48, torch.float32)
    _cuda_ok()
    _check_unsort(got.xs, got.pos, None, torch.float32)
    dxs = torch.randn(240, 48, generator=torch.Generator().manual_seed(1)).cuda()
    dx = sp.moe_sort_backward(dxs, got.pos)
    assert torch.equal(dx, sp.moe_unsort(dxs, got.pos))
    # against differences: xs is linear in x, so L = sum dxs * xs moves by dx exactly
    live = int(got.offsets[-1])
    ref = torch.zeros(60, 48, dtype=torch.float64)
    ref.index_add_(0, got.src[:live].cpu().long() // 4, dxs[:live].double().cpu())
    mag = torch.zeros(60, 48, dtype=torch.float64)
    mag.index_add_(0, got.src[:live].cpu().long() // 4, dxs[:live].double().abs().cpu())
    assert ((dx.double().cpu() - ref).abs() <= 5 * U * mag).all()
    d, dw = sp.moe_unsort_backward(dx, got.xs, got.pos)
    assert dw is None and (d[live:] == 0).all()


def test_unsort_bad_rows_are_empty_and_reported():
    ys = torch.ones(6, 8, device="cuda")
    pos = torch.tensor([[0, 6], [-1, 3], [-7, 5]], dtype=torch.int32, device="cuda")
    w = torch.ones(3, 2, device="cuda")
    _check_unsort(ys, pos, w, torch.float32)
    assert sp.last_device_error() == sp.ERR_INVALID_ARG
    # fewer rows than entries: the rows behind the last expert need not exist
    y = sp.moe_unsort(ys[:4], torch.tensor([[0, 3], [-1, -1]], dtype=torch.int32, device="cuda"))
    _cuda_ok()
    assert y[:, 0].tolist() == [2.0, 0.0]


def test_unsort_infinities_stay_in_their_tokens():
    ys = torch.ones(4, 16, device="cuda")
    ys[2] = float("inf")
    pos = torch.tensor([[0, 1], [2, 3]], dtype=torch.int32, device="cuda")
    y = sp.moe_unsort(ys, pos, torch.full((2, 2), 0.5, device="cuda"))
    assert (y[0] == 1).all() and torch.isinf(y[1]).all()


def test_unsort_offsets_beyond_32_bits():
    """rows * H above 2^31 elements: the last rows are where they should be."""
    H, rows = 32776, 65540
    ys = torch.zeros(rows, H, dtype=torch.bfloat16, device="cuda")
    ys[-1] = 3.0
    ys[-2] = 5.0
    pos = torch.tensor([[rows - 1, rows - 2]], dtype=torch.int32, device="cuda")
    w = torch.tensor([[2.0, 0.5]], device="cuda")
    y = sp.moe_unsort(ys, pos, w)
    assert (y == 8.5).all()
    dys, dw = sp.moe_unsort_backward(y, ys, pos, w)
    _cuda_ok()
    assert (dys[-1] == 17.0).all() and (dys[-2] == 4.25).all() and not dys[:-2].any()
    assert dw.tolist() == [[8.5 * 3 * H, 8.5 * 5 * H]]


def test_sort_rows_beyond_32_bits():
    T, k, H = 16400, 4, 32776
    x = torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = (torch.arange(T, device="cuda") % 97).bfloat16()
    r = torch.randint(0, 4, (T, k), generator=torch.Generator().manual_seed(1)).int().cuda()
    got = sp.moe_sort(x, r, 4)
    _cuda_ok()
    assert torch.equal(got.xs[:, 0], x[(got.src // k).long(), 0])


# ------------------------------------------------------------------------------------ how it is called

def test_refusals():
    x = torch.zeros(4, 16, device="cuda")
    ids = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    for call, err in ((lambda: sp.moe_route(x[:, ::2], 2), ValueError), (lambda: sp.moe_route(x.double(), 2), TypeError),
                      (lambda: sp.moe_route(x[0], 2), ValueError), (lambda: sp.moe_route(x, 17), sp.SP24Error),
                      (lambda: sp.moe_sort(x, ids.long(), 4), TypeError), (lambda: sp.moe_sort(x[:3], ids, 4), ValueError),
                      (lambda: sp.moe_sort(x, ids.cpu(), 4), ValueError), (lambda: sp.moe_sort(x, ids, 0), sp.SP24Error),
                      (lambda: sp.moe_unsort(x, ids, torch.zeros(4, 3, device="cuda")), ValueError),
                      (lambda: sp.moe_unsort(x.bfloat16(), ids, dtype=torch.float16), sp.SP24Error),
                      (lambda: sp.moe_unsort(x, ids, out=torch.zeros(4, 15, device="cuda")), ValueError),
                      (lambda: sp.moe_unsort_backward(x[:3], x, ids), ValueError),
                      (lambda: sp.moe_route_backward(x, x, ids), ValueError)):
        with pytest.raises(err):
            call()


@pytest.mark.parametrize("T", [300, 2500])
def test_other_stream_and_graph(T):
    """On a stream of its own, and captured and replayed on new inputs: the results of plain calls."""
    g = torch.Generator().manual_seed(9)
    E, k, H = 40, 4, 96
    logits = torch.randn(T, E, generator=g).cuda()
    x = torch.randn(T, H, generator=g).bfloat16().cuda()

    def chain(stream=None):
        routing, w = sp.moe_route(logits, k, stream=stream)
        s = sp.moe_sort(x, routing, E, stream=stream)
        y = sp.moe_unsort(s.xs, s.pos, w, stream=stream)
        dys, dw = sp.moe_unsort_backward(y, s.xs, s.pos, w, stream=stream)
        return [routing, w, *s, y, dys, dw, sp.moe_sort_backward(dys, s.pos, stream=stream),
                sp.moe_route_backward(dw, logits, routing, stream=stream)]

    want = chain()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = chain(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = chain()
    logits.copy_(torch.randn(T, E, generator=g))
    x.copy_(torch.randn(T, H, generator=g))
    graph.replay()
    again = [t.clone() for t in held]
    assert all(torch.equal(a, b) for a, b in zip(again, chain()))
    _cuda_ok()


def test_sorts_at_once_on_two_streams():
    """Sorts that overlap, each with a workspace of its own."""
    rs = [torch.from_numpy(np.random.default_rng(s).integers(0, 30, (3000, 3)).astype(np.int32)).cuda() for s in range(2)]
    want = [sp.moe_sort_tables(r, 30) for r in rs]
    streams = [torch.cuda.Stream() for _ in rs]
    torch.cuda.synchronize()
    got = [(i, sp.moe_sort_tables(rs[i], 30, stream=streams[i])) for _ in range(20) for i in range(2)]
    _cuda_ok()
    assert all(torch.equal(a, b) for i, t in got for a, b in zip(t[1:], want[i][1:]))


@pytest.mark.parametrize("T", [100, 1500, 12000])
def test_calls_without_a_wait_between(T):
    """Each call starts while the one before it ends: what it reads has to be written all the same."""
    g = torch.Generator().manual_seed(T)
    E, k, H = 64, 4, 64
    logits = [torch.randn(T, E, generator=g).cuda() for _ in range(4)]
    x = torch.randn(T, H, generator=g).cuda()

    def step(l, wait):
        routing, w = sp.moe_route(l, k)
        if wait:
            torch.cuda.synchronize()
        s = sp.moe_sort(x, routing, E)
        if wait:
            torch.cuda.synchronize()
        y = sp.moe_unsort(s.xs, s.pos, w)
        if wait:
            torch.cuda.synchronize()
        dys, dw = sp.moe_unsort_backward(y, s.xs, s.pos, w)
        if wait:
            torch.cuda.synchronize()
        return [routing, *s, y, dys, dw, sp.moe_route_backward(dw, l, routing)]

    want = [step(l, True) for l in logits]
    got = [step(logits[i % 4], False) for i in range(24)]
    _cuda_ok()
    for i, r in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(r, want[i % 4]))


def test_route_weights_of_one_expert_and_extremes():
    """One expert; logits at the type's ends (differences that overflow to infinity included)."""
    l = torch.tensor([[3.0e38, -3.0e38, 1.0, 3.0e38], [-3.0e38, -3.0e38, -3.0e38, -3.0e38]], device="cuda")
    ids, w = sp.moe_route(l, 2)
    assert ids.tolist() == [[0, 3], [0, 1]] and w.tolist() == [[0.5, 0.5], [0.5, 0.5]]
    _, w = sp.moe_route(l, 2, sp.ROUTE_SIGMOID, False)
    assert w.tolist() == [[1.0, 1.0], [0.0, 0.0]]
    ids, w = sp.moe_route(l, 2, sp.ROUTE_SIGMOID, True)  # a sum of 0 leaves weights of 0
    assert w.tolist() == [[0.5, 0.5], [0.0, 0.0]]
    d = sp.moe_route_backward(torch.ones(2, 2, device="cuda"), l, ids, sp.ROUTE_SIGMOID, True)
    assert not d.any()
    ids, w = sp.moe_route(l[:, :1].contiguous(), 1, sp.ROUTE_SOFTMAX, False)
    assert ids.tolist() == [[0], [0]] and w.tolist() == [[1.0], [1.0]]


def _off(rows, H, dtype, off, fill=None, seed=0):
    """[rows, H] that starts `off` elements behind a 256-byte boundary, and the buffer it lies in."""
    flat = torch.full((rows * H + off + 16,), 7.0, dtype=dtype, device="cuda")
    view = flat[off:off + rows * H].view(rows, H)
    if fill is None:
        view.copy_(torch.randn(rows, H, generator=torch.Generator().manual_seed(seed)))
    return view, flat


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,k,H,a,b", [(1, 1, 1, 1, 0), (1, 1, 9, 3, 5), (5, 3, 17, 0, 1), (40, 2, 47, 7, 2), (700, 4, 16, 0, 0),
                                       (701, 3, 24, 0, 4), (900, 3, 33, 1, 1), (1100, 2, 250, 2, 0), (690, 3, 255, 5, 6),
                                       (1030, 2, 1001, 0, 3), (3, 2, 4099, 1, 4), (2100, 1, 8, 1, 0)])
def test_sort_rows_of_every_start(dtype, T, k, H, a, b):
    """Rows and tensors that start anywhere, in one launch and in three; nothing beside the rows is written."""
    x, _ = _off(T, H, dtype, a)
    xs, around = _off(T * k, H, dtype, b, fill=7)
    rng = np.random.default_rng(H)
    r = torch.from_numpy(rng.integers(-1, 9, (T, k)).astype(np.int32)).cuda()
    i32 = lambda *s: torch.empty(s, dtype=torch.int32, device="cuda")  # noqa: E731
    got = sp.moe_sort(x, r, 9, out=(xs, i32(T, k), i32(T * k), i32(T * k), i32(10)))
    want = torch.full_like(around, 7.0)
    live = int(got.offsets[-1])
    want[b:b + live * H] = x[(got.src[:live] // k).long()].reshape(-1)
    assert torch.equal(around, want)
    _cuda_ok()


@pytest.mark.parametrize("pair", PAIRS, ids=lambda p: "-".join(str(d)[6:] for d in p))
@pytest.mark.parametrize("T,k,H,a,b,c", [(1, 1, 1, 1, 0, 2), (2, 3, 9, 3, 5, 0), (5, 2, 16, 0, 0, 0), (9, 6, 17, 0, 1, 1),
                                         (30, 2, 47, 7, 2, 4), (33, 7, 24, 0, 4, 8), (20, 5, 33, 1, 1, 1), (21, 3, 250, 2, 0, 6),
                                         (7, 4, 255, 5, 6, 3), (5, 2, 1001, 0, 3, 2), (4, 6, 1001, 4, 0, 1), (2, 3, 4099, 1, 4, 5)])
def test_unsort_rows_of_every_start(pair, T, k, H, a, b, c):
    """The rows of ys, y, dy and dys start anywhere; nothing beside them is written."""
    g = torch.Generator().manual_seed(T + H)
    pos = torch.randperm(T * k, generator=g).int().view(T, k)
    pos[T // 2, k - 1] = -1
    w = torch.rand(T, k, generator=g)
    pos, w = pos.cuda(), w.cuda()
    ys, _ = _off(T * k, H, pair[0], a, seed=1)
    y, y_around = _off(T, H, pair[1], b, fill=7)
    dy, _ = _off(T, H, pair[1], c, seed=2)
    dys, dys_around = _off(T * k, H, pair[0], b, fill=7)
    # what aligned tensors of the same values give: the sums run in the same order, slot by slot
    want = sp.moe_unsort(_whole(ys), pos, w, dtype=pair[1])[:, :H]
    assert torch.equal(sp.moe_unsort(ys, pos, w, out=y), want)
    live = pos[pos >= 0].long()
    ref_dys = torch.full_like(ys, 7.0)
    ref_dys[live] = (w[..., None] * dy[:, None].float())[pos >= 0].to(pair[0])
    dw = torch.full((T, k), 7.0, device="cuda")
    sp.moe_unsort_backward(dy, ys, pos, w, out=(dys, dw))
    assert torch.equal(dys, ref_dys)
    # a dot product of H terms in any order
    terms = (dy[:, None].double() * ys.double()[pos.clamp(min=0).long()]) * (pos >= 0)[..., None]
    assert ((dw.double() - terms.sum(2)).abs() <= (H + 1) * U * terms.abs().sum(2) + TINY[torch.float32]).all()
    alone, alone_around = _off(T * k, H, pair[0], a, fill=7)
    sp.moe_unsort_backward(dy, ys, pos, w, out=(alone, None))
    assert torch.equal(alone, ref_dys)
    for view, flat, b in ((y, y_around, b), (dys, dys_around, b), (alone, alone_around, a)):
        edge = flat.clone()
        edge[b:b + view.numel()] = 7.0
        assert (edge == 7.0).all()
    _cuda_ok()


def _whole(t):
    """t in rows of a multiple of 16 elements."""
    return torch.nn.functional.pad(t, (0, -t.shape[1] % 16)).contiguous()
