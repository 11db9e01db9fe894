"""Serving attention on the GPU with values at the border of what can be
weighed: infinite V behind scores that are far apart."""
import pytest
import torch

from serving_cases import DTYPES, paged_batch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from long_context_blockwise_max_b200 import serving
    assert torch.cuda.is_available()
    return serving


def ok(S, ws):
    from long_context_blockwise_max_b200 import pulsar
    return pulsar.pa_workspace_status(ws)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("q_len,kv_len", [(1, 900), (2, 700), (4, 1000), (1, 9000), (2, 9000), (4, 20000), (40, 9000),
                                          (70, 300), (1, 100), (150, 9000)])
def test_a_visible_infinity_with_a_vanishing_weight_is_not_lost(S, dtype, q_len, kv_len):
    # scores 0 but for the last keys that every row sees, whose scores are 128:
    # the first keys weigh exp(-128), which is zero in fp32, and they are in
    # another part when the keys are cut.  A column with a non-finite V that a
    # row sees is non-finite all the same, cut or not; the others are as without.
    dt = DTYPES[dtype]
    c = paged_batch([q_len], [kv_len], 8, 2, 64, 16, dt, seed=kv_len, poison=False)
    q = torch.full_like(c["q"], 4.0)
    k, v = torch.zeros_like(c["k_pages"]), c["v_pages"].clone()
    page = lambda key: (int(c["table"][0, key // 16]), key % 16)
    for key in range(kv_len - q_len - 6, kv_len - q_len):
        k[page(key)] = 4.0
    args = (q, c["cu_q"], c["kv_len"], c["table"], k)
    o0, lse0, ws = S.pa_paged_attend(*args, v, q_len)
    assert ok(S, ws) == 0 and torch.isfinite(o0).all() and torch.isfinite(lse0).all()
    v[page(0)][0, 5], v[page(1)][0, 6], v[page(2)][1, 7] = float("inf"), -float("inf"), float("nan")
    o, lse, ws = S.pa_paged_attend(*args, v, q_len)
    assert ok(S, ws) == 0 and torch.equal(lse, lse0)
    assert not torch.isfinite(o[:, :4, 5:7]).any() and not torch.isfinite(o[:, 4:, 7]).any()
    keep = torch.ones_like(o, dtype=torch.bool)
    keep[:, :4, 5:7] = False
    keep[:, 4:, 7] = False
    assert torch.equal(o[keep], o0[keep])
