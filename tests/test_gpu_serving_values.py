"""Serving attention on the GPU with values at the border of what can be
weighed or counted: infinite V behind scores that are far apart, scores of
-inf, caches as long as a table allows, K and V too large for L2 (another order
of work)."""
import numpy as np
import pytest
import torch

from oracle import serving_oracle as so
from serving_cases import DTYPES, check_rows, half_step, paged_batch, randn

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


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("q_len,kv_len", [(1, 60), (1, 9000), (4, 9000), (40, 300), (40, 9000), (150, 400)])
def test_scores_of_minus_infinity(S, dtype, q_len, kv_len):
    # a key whose score is -inf weighs nothing; a row all of whose keys are such
    # counts as one that sees no key, whichever kernel has it
    c = paged_batch([q_len], [kv_len], 8, 2, 64, 16, DTYPES[dtype], seed=q_len, poison=False)
    q, k = c["q"].abs() + 0.5, c["k_pages"].clone()
    args = lambda k: (q, c["cu_q"], c["kv_len"], c["table"], k, c["v_pages"], q_len)
    k[:, :, 0] = -float("inf")
    o, lse, ws = S.pa_paged_attend(*args(k))
    assert ok(S, ws) == 0
    assert (o[:, :4] == 0).all() and torch.isneginf(lse[:, :4]).all()
    o0, lse0, _ = S.pa_paged_attend(*args(c["k_pages"]))
    assert torch.equal(o[:, 4:], o0[:, 4:]) and torch.equal(lse[:, 4:], lse0[:, 4:])
    # all but the first key: every row's answer is its V
    page = int(c["table"][0, 0])
    k[page, 0, 0] = 0.0
    o, lse, ws = S.pa_paged_attend(*args(k))
    assert ok(S, ws) == 0 and (lse[:, :4] == 0).all()
    assert (o[:, :4] == c["v_pages"][page, 0, 0]).all()


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


def test_a_piece_may_last_longer_than_a_wait_between_tiles(S):
    # more kv heads than cuts are made for: each piece has all of 200 million keys,
    # 1.8 s of work.  Equal scores.
    hkv, d, page, width, m = 152, 64, 1024, 200_000, 20
    k = torch.zeros((1, page, hkv, d), dtype=torch.bfloat16, device="cuda")
    v = torch.ones_like(k)
    q = torch.ones((m, hkv, d), dtype=torch.bfloat16, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    table = torch.zeros((1, width), dtype=torch.int32, device="cuda")
    o, lse, ws = S.pa_paged_attend(q, i32([0, m]), i32([width * page]), table, k, v, m)
    assert ok(S, ws) == 0
    assert torch.isfinite(o).all()
    keys = torch.arange(width * page - m + 1, width * page + 1, dtype=torch.float64)
    assert (lse.double().cpu() - keys.log()[:, None]).abs().max() <= 1e-4


# What the tensor core adds in one accumulator: 2048 tiles of 128 keys, 16 keys to an
# addition that drops the bits below its sum's last place, 2^-23 each at most.
LONG_SUM = 2048 * 8 * 2.0 ** -23


@pytest.mark.parametrize("kind,n_keys", [("one row tile", 2 ** 23), ("two row tiles", 2 ** 22), ("cut", 2 ** 27),
                                         ("ragged", 2 ** 22 + 2048 * 128 + 1), ("one token", 2 ** 27),
                                         ("one token, 16 rows", 2 ** 27), ("two tokens, 12 rows", 2 ** 26)])
def test_sums_over_millions_of_keys_keep_their_size(S, kind, n_keys):
    # equal scores: o is the mean of V over the keys, whatever their number.  (With
    # 152 kv heads the keys are not cut.)
    hq, hkv, m = {"one row tile": (152, 152, 20), "two row tiles": (608, 152, 64), "cut": (32, 8, 64),
                  "ragged": (608, 152, 61), "one token": (8, 8, 1), "one token, 16 rows": (128, 8, 1),
                  "two tokens, 12 rows": (48, 8, 2)}[kind]
    page, d = 1024, 64
    width = -(-n_keys // page)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    k = torch.zeros((1, page, hkv, d), dtype=torch.bfloat16, device="cuda")
    q = torch.ones((m, hq, d), dtype=torch.bfloat16, device="cuda")
    args = (q, i32([0, m]), i32([n_keys]), torch.zeros((1, width), dtype=torch.int32, device="cuda"), k)
    o, lse, ws = S.pa_paged_attend(*args, torch.ones_like(k), m)
    assert ok(S, ws) == 0 and (o == 1).all()
    assert (lse[-1].double() - np.log(n_keys)).abs().max() <= 1e-4
    v = (randn(k.shape, torch.float32, 90).abs() + 0.5).bfloat16()
    o, lse, ws = S.pa_paged_attend(*args, v, m)
    assert ok(S, ws) == 0
    # (whole pages but for less than 2^-11 of the keys)
    want = v[0].double().mean(0).repeat_interleave(hq // hkv, 0)
    off = (o[-1].double() - want) / want
    assert off.abs().max() <= half_step(torch.bfloat16) + LONG_SUM + 2.0 ** -11
    assert off.mean().abs() <= LONG_SUM


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1, 3], [700, 1, 2000]), ([40, 1, 200], [300, 900, 3000]), ([100], [9000]),
                                            ([1, 2, 1], [0, 5, 129]), ([300, 20, 0, 7], [300, 20, 4, 500])])
def test_a_wide_table_changes_no_result(S, d, q_lens, kv_lens):
    # the same requests in a table with room for more than a million keys each: the
    # kernels that can fold, with nothing to fold
    c = paged_batch(q_lens, kv_lens, 16, 4, d, 16, torch.bfloat16, seed=d + len(q_lens))
    run = lambda t: S.pa_paged_attend(c["q"], c["cu_q"], c["kv_len"], t, c["k_pages"], c["v_pages"], c["max_q"])
    o0, lse0, ws = run(c["table"])
    assert ok(S, ws) == 0
    wide = torch.full((len(q_lens), 70_000), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    wide[:, :c["table"].shape[1]] = c["table"]
    o, lse, ws2 = run(wide)
    assert ok(S, ws2) == 0 and torch.equal(lse, lse0) and torch.equal(o, o0)


def test_a_prompt_longer_than_one_sum(S):
    # 600K tokens, more than two sums; scores grow along the sequence, so that the
    # running maximum passes what was added before; then an infinite V near the front
    n, hq, hkv, d = 600_000, 4, 1, 64
    q, k = randn((n, hq, d), torch.bfloat16, 91), randn((n, hkv, d), torch.float32, 92)
    k = (k * torch.linspace(0.2, 3.0, n, device="cuda")[:, None, None]).bfloat16()
    v = (randn((n, hkv, d), torch.float32, 93).abs() + 0.5).bfloat16()
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    o, lse, ws = S.pa_prompt_attend(q, k, v, cu)
    assert ok(S, ws) == 0 and torch.isfinite(o).all()
    # (64 bits on the GPU: the rows have up to 600K keys)
    kd, vd = k[:, 0].double(), v[:, 0].double()
    half = half_step(torch.bfloat16)
    for i in (0, 2047 * 128, 2048 * 128 - 1, 2048 * 128, 2048 * 128 + 64, 400_000, 2 * 2048 * 128 + 5, n - 1):
        s = q[i].double() @ kd[:i + 1].T / d ** 0.5
        z = torch.logsumexp(s, -1)
        want = torch.exp(s - z[:, None]) @ vd[:i + 1]
        # P rounded, o rounded, and the sum (V is positive: sum p |v| = o)
        off = ((o[i].double() - want) / want).abs().max()
        assert off <= 2 * half * (1 + half) + LONG_SUM, f"row {i}: {off:.2e}"
        assert (lse[i].double() - z).abs().max() <= 1e-4, f"row {i}"
    v2 = v.clone()
    v2[1000, 0, 5] = float("inf")
    o2, lse2, ws = S.pa_prompt_attend(q, k, v2, cu)
    assert ok(S, ws) == 0 and torch.equal(lse2, lse)
    assert not torch.isfinite(o2[1000:, :, 5]).any()
    keep = torch.ones_like(o, dtype=torch.bool)
    keep[1000:, :, 5] = False
    assert torch.equal(o2[keep], o[keep])


def spread_rows(n, count):
    """The ends of a sequence, and rows of it at about equal distances."""
    return sorted({0, n - 1} | {int(x) for x in np.linspace(0, n - 1, count)})


@pytest.mark.parametrize("lens", [[32768], [20001, 9000, 1, 5000]], ids=["one", "several"])
def test_prompts_beyond_the_cache(S, lens):
    # 134 MB and more of K and V in more than two waves of pieces per kv head:
    # the pieces of one kv head run together, where shorter calls take all heads
    # in order of depth.  Rows spread over each prompt against 64 bits.
    n, hq, hkv, d = sum(lens), 32, 8, 128
    q, k, v = (randn((n, h, d), torch.bfloat16, 70 + i) for i, h in enumerate((hq, hkv, hkv)))
    cu = np.concatenate([[0], np.cumsum(lens)])
    o, lse, ws = S.pa_prompt_attend(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"))
    assert ok(S, ws) == 0 and torch.isfinite(o).all() and torch.isfinite(lse).all()
    for b, m in enumerate(lens):
        kh, vh = (t[cu[b]:cu[b + 1]].double().cpu().numpy() for t in (k, v))
        for i in spread_rows(m, 8):
            row = slice(cu[b] + i, cu[b] + i + 1)
            want = so.attend_rows(q[row].double().cpu().numpy(), kh[:i + 1], vh[:i + 1], i)
            check_rows(torch.bfloat16, o[row], lse[row], want, i + 1, f"prompt {b}, row {i}")


def test_paged_chunks_beyond_the_cache(S):
    # the same order of work over pages: two chunks behind long caches
    q_lens, kv_lens, hq, hkv, d = [9000, 12000], [20000, 17000], 32, 8, 128
    page, n = 64, 21000
    n_pages = sum(-(-kv // page) for kv in kv_lens)
    k, v = (randn((n_pages, page, hkv, d), torch.bfloat16, 80 + i) for i in range(2))
    q = randn((n, hq, d), torch.bfloat16, 82)
    order = np.random.default_rng(8).permutation(n_pages)
    table = np.zeros((2, max(-(-kv // page) for kv in kv_lens)), dtype=np.int64)
    at = 0
    for b, kv in enumerate(kv_lens):
        held = -(-kv // page)
        table[b, :held] = order[at:at + held]
        at += held
    i32 = lambda x: torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")
    o, lse, ws = S.pa_paged_attend(q, i32([0, 9000, 21000]), i32(kv_lens), i32(table), k, v, 12000)
    assert ok(S, ws) == 0 and torch.isfinite(o).all() and torch.isfinite(lse).all()
    kh, vh = (t.float().cpu().numpy() for t in (k, v))
    for b, (m, kv) in enumerate(zip(q_lens, kv_lens)):
        keys, vals = (so.paged_keys(x, table[b], kv).astype(np.float64) for x in (kh, vh))
        lo = 9000 * b
        for i in spread_rows(m, 6):
            row, seen = slice(lo + i, lo + i + 1), kv - m + i + 1
            want = so.attend_rows(q[row].double().cpu().numpy(), keys[:seen], vals[:seen], seen - 1)
            check_rows(torch.bfloat16, o[row], lse[row], want, seen, f"chunk {b}, row {i}")
