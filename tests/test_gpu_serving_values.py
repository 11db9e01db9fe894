"""Serving attention on the GPU with values at the border of what can be
weighed or counted: infinite V behind scores that are far apart, caches as
long as a table allows."""
import pytest
import torch

from oracle import serving_oracle as so
from serving_cases import DTYPES, check_rows, paged_batch

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


@pytest.mark.parametrize("q_lens", [[1, 1, 2], [3, 1, 40]], ids=["decode", "chunk"])
def test_a_cache_as_long_as_a_table_allows(S, q_lens):
    # 2^31 - 16 keys: one page of zeros, many times over, then one of ordinary
    # keys, whose scores weigh by e^40 more than all the others.  The long request
    # comes last, behind short ones.
    hq, hkv, d, page = 8, 1, 64, 16
    width = (2 ** 31 - 1) // page
    kv_lens = [5, 0, width * page]
    table = torch.zeros((3, width), dtype=torch.int32, device="cuda")
    table[2, -4:] = torch.arange(1, 5, device="cuda")
    table[0, 0] = 5
    k, v = (torch.zeros((6, page, hkv, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    gen = torch.Generator().manual_seed(4)
    k[1:, :, :, 0] = 64.0      # 64 * 8 / sqrt(64) = 64 above the zeros' score; 2^31 of them weigh e^(21.5 - 64)
    k[1:] += torch.randn((5, page, hkv, d), generator=gen).to(k)
    v[1:] = torch.randn((5, page, hkv, d), generator=gen).to(v)
    n = sum(q_lens)
    q = torch.randn((n, hq, d), generator=gen).to(v)
    q[:, :, 0] = 8.0
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    cu = torch.tensor([0, q_lens[0], q_lens[0] + q_lens[1], n], dtype=torch.int32, device="cuda")
    kv = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")
    o, lse, ws = S.pa_paged_attend(q, cu, kv, table, k, v, max(q_lens))
    assert ok(S, ws) == 0
    qh, kh, vh = (t.double().cpu().numpy() for t in (q, k, v))
    at = 0
    for b, (m, row, keys) in enumerate(zip(q_lens, ([5], [], [1, 2, 3, 4]), (5, 0, 64))):
        if m and keys:
            kk, vv = (x[row].reshape(-1, hkv, d)[:keys] for x in (kh, vh))
            want = so.attend_rows(qh[at:at + m], kk, vv, keys - m)
            check_rows(torch.bfloat16, o[at:at + m], lse[at:at + m], want, keys, f"request {b}")
        elif m:
            assert (o[at:at + m] == 0).all() and torch.isneginf(lse[at:at + m]).all()
        at += m
