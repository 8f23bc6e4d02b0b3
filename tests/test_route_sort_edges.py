"""What valid calls of the router, the sort and the unsort leave in the device error word: nothing."""
import numpy as np
import pytest
import torch

import fp16_gemm_b200 as sp
from test_parity_route_sort import DTYPES, FORMS, _check_sort, _cuda_ok

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES, ids=["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,k,E,H", [(1, 1, 1, 1), (1, 2, 3, 8), (8, 10, 512, 64), (33, 3, 7, 129), (100, 4, 16, 2),
                                     (257, 2, 5, 40), (64, 8, 64, 1000), (300, 10, 40, 16), (1000, 7, 333, 24),
                                     (9000, 1, 30000, 3), (2049, 1, 2, 16)])
def test_a_valid_sort_reports_nothing(dtype, T, k, E, H):
    """Ids over the whole range, the first and the last expert and empty slots among them, in one launch
    and in four."""
    _cuda_ok()
    r = np.random.default_rng(T + E).integers(-1, E, (T, k)).astype(np.int32)
    r.flat[0], r.flat[-1] = E - 1, 0
    _check_sort(r, E, H, dtype)
    _cuda_ok()


@pytest.mark.parametrize("form", FORMS, ids=["softmax_renorm", "softmax", "sigmoid_renorm", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(5, 3, 3), (70, 64, 8), (3000, 100, 4)])
def test_a_valid_round_reports_nothing(form, T, E, k):
    """Router, sort, unsort and all gradients on a batch with masked tokens and masked experts."""
    _cuda_ok()
    l = torch.randn(T, E, generator=torch.Generator().manual_seed(T))
    l[T - T // 4 - 1:] = -float("inf")
    l[0, 1:] = -float("inf")
    l = l.cuda()
    routing, w = sp.moe_route(l, k, *form)
    s = sp.moe_sort(l, routing, E)
    y = sp.moe_unsort(s.xs, s.pos, w)
    dys, dw = sp.moe_unsort_backward(torch.ones_like(y), s.xs.nan_to_num(0.0, 0.0, 0.0), s.pos, w)
    sp.moe_sort_backward(dys, s.pos)
    d = sp.moe_route_backward(dw, l, routing, *form)
    _cuda_ok()
    assert torch.isfinite(d).all() and not d[T - T // 4 - 1:].any()
