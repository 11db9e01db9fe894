"""Serving operators on the GPU against the fp64 / integer oracle: page
tables and slot maps, rotate-and-append, packed prompt attention, paged
attention, and a whole step of them in the order of use."""
import os
import subprocess
import sys
import threading

import numpy as np
import pytest
import torch

import oracle
from oracle import serving_oracle as so
from serving_cases import (DTYPES, bounds, check_paged, check_rows, half_step, paged_batch, randn)

pytestmark = pytest.mark.gpu

HEADS = [(32, 8), (4, 2), (8, 8), (28, 4), (5, 1), (16, 1), (64, 1)]


@pytest.fixture(scope="module")
def S():
    from long_context_blockwise_max_b200 import serving
    assert torch.cuda.is_available()
    return serving


def ok(S, ws):
    from long_context_blockwise_max_b200 import pulsar
    return pulsar.pa_workspace_status(ws)


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ schedule
@pytest.mark.parametrize("B,page,q_hi,kv_hi,extra", [(1, 16, 1, 100, 0), (7, 16, 40, 100, 5), (64, 64, 1, 5000, 0),
                                                     (1024, 16, 3, 300, 11), (1025, 32, 70, 2000, 1), (3, 256, 5000, 10, 0),
                                                     (8192, 16, 2, 20, 0)])
def test_schedule_matches_the_oracle(S, B, page, q_hi, kv_hi, extra):
    rng = np.random.default_rng(B + page)
    q, kv = rng.integers(0, q_hi + 1, B), rng.integers(0, kv_hi + 1, B)
    held = -(-kv // page)
    width = int((-(-(kv + q) // page)).max()) + 2
    pool = rng.permutation(int(held.sum() + (-(-(kv + q) // page)).sum()) + 4)
    table = np.full((B, width), -5, dtype=np.int64)
    at = 0
    for b in range(B):
        table[b, :held[b]] = pool[at:at + held[b]]
        at += held[b]
    free = pool[at:]
    n = int(q.sum()) + extra
    cu, kv_out, pos, slots, used, tab, refused = so.schedule_step(q, kv, table, free, page, n)
    assert not refused
    wide = i32(np.concatenate([table, np.full((B, 3), -9)], 1))
    t = wide[:, :width]                       # rows of a wider table
    got = S.pa_paged_schedule(i32(q), i32(kv), t, i32(free), page, n)
    assert ok(S, got[-1]) == 0
    for name, g, w in zip(("cu_q", "kv_len", "positions", "slots", "used"), got, (cu, kv_out, pos, slots, [used])):
        assert np.array_equal(g.cpu().numpy(), w), name
    assert np.array_equal(t.cpu().numpy(), tab)
    assert (wide[:, width:] == -9).all()


def test_schedule_refuses_whole_requests(S):
    from long_context_blockwise_max_b200 import pulsar
    # request 1 does not fit its table row, request 3 the pool; 4 needs no
    # page and is granted, 5 needs one and is refused with the pool asked out
    q, kv, page = [10, 200, 16, 100, 2, 16], [0, 20, 16, 0, 3, 0], 16
    table = np.full((6, 4), -1, dtype=np.int64)
    table[1, :2], table[2, 0], table[4, 0] = [50, 51], 52, 53
    q[3] = 60                                  # four pages: fits a row, not the pool
    free = np.array([7, 3, 9])
    n = sum(q)
    cu, kv_out, pos, slots, used, tab, refused = so.schedule_step(q, kv, table, free, page, n)
    assert refused == [1, 3, 5] and used == 2
    t = i32(table)
    got = S.pa_paged_schedule(i32(q), i32(kv), t, i32(free), page, n)
    assert ok(S, got[-1]) == -7
    for g, w in zip(got, (cu, kv_out, pos, slots, [used])):
        assert np.array_equal(g.cpu().numpy(), w)
    assert np.array_equal(t.cpu().numpy(), tab)
    prev = pulsar.set_status_checks(True)
    try:
        with pytest.raises(pulsar.PulsarError) as e:
            S.pa_paged_schedule(i32(q), i32(kv), i32(table), i32(free), page, n)
        assert e.value.code == -7
    finally:
        pulsar.set_status_checks(prev)


def test_schedule_records_invalid_lengths(S):
    t = i32(np.zeros((2, 4)))
    got = S.pa_paged_schedule(i32([-3, 5]), i32([0, 0]), t, i32([4]), 16, 5)
    assert ok(S, got[-1]) == -1
    assert got[0].tolist() == [0, 0, 5] and got[3].tolist() == [64, 65, 66, 67, 68]
    got = S.pa_paged_schedule(i32([4, 5]), i32([0, 0]), t, i32([4, 1]), 16, 6)     # 9 tokens, room for 6
    assert ok(S, got[-1]) == -1
    assert got[3].tolist() == [64, 65, 66, 67, 16, 17]
    got = S.pa_paged_schedule(i32([2]), i32([0]), t[:1], i32([2 ** 31 - 1]), 16, 2)  # slots past 2^31
    assert ok(S, got[-1]) == -1 and got[3].tolist() == [-1, -1]


# -------------------------------------------------------------------- append
@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("N,hq,hkv,base,theta", [(1, 32, 8, 131072, 5e5), (5, 4, 2, 0, 1e4), (37, 28, 4, 1 << 20, 5e5),
                                                 (1200, 5, 1, 7, 1e4), (3, 8, 8, 2 ** 31 - 5, 1e4)])
def test_append_matches_the_oracle(S, dtype, d, N, hq, hkv, base, theta):
    dt = DTYPES[dtype]
    page, n_pages = 16, -(-N // 16) + 2
    fused = randn((N, hq + 2 * hkv, d), dt, seed=N + d)
    q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    pos = base + np.arange(N)
    rng = np.random.default_rng(N)
    slots = rng.permutation(n_pages * page)[:N]
    slots[::3] = -1
    kp = torch.full((n_pages, page, hkv, d), 7.0, dtype=dt, device="cuda")
    vp = kp.clone()
    qo, ko, ws = S.pa_paged_append(q, k, v, i32(pos), i32(slots), kp, vp, rope_theta=theta, want_k=True)
    assert ok(S, ws) == 0
    # cos and sin are off by 2^-24 (rounding) + 2^-22 (angle: a turn's fraction in
    # fp32 is off by 2^-26 turns, 2 pi * 2^-26 < 2^-23, and the function by 2^-23);
    # two products and a sum in fp32 of values up to |x1| + |x2|, then one rounding
    def near(got, want, x, what):
        xs = np.abs(x.double().cpu().numpy())
        half = d // 2
        size = np.concatenate([xs[..., :half] + xs[..., half:]] * 2, -1)
        err = np.abs(got.double().cpu().numpy() - want)
        fp = 2.0 ** -20 * size
        assert (err <= fp + half_step(dt) * (np.abs(want) + fp)).all(), what
    near(qo, so.rope(q.double().cpu().numpy(), pos, theta), q, "q")
    near(ko, so.rope(k.double().cpu().numpy(), pos, theta), k, "k")
    kf, vf = kp.view(-1, hkv, d), vp.view(-1, hkv, d)
    put = slots >= 0
    at = torch.from_numpy(slots[put]).cuda()
    assert torch.equal(kf[at], ko[torch.from_numpy(put).cuda()])
    assert torch.equal(vf[at], v[torch.from_numpy(put).cuda()])
    rest = torch.ones(n_pages * page, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert (kf[rest] == 7).all() and (vf[rest] == 7).all()


def test_append_in_place_without_pages_and_without_rotation(S):
    q, k, v = randn((9, 8, 64), torch.bfloat16, 1), randn((9, 2, 64), torch.bfloat16, 2), randn((9, 2, 64), torch.bfloat16, 3)
    pos = i32(np.arange(9) * 1000)
    want_q, want_k, _ = S.pa_paged_append(q, k, None, pos, None, None, None, rope_theta=1e4, want_k=True)
    q2, k2 = q.clone(), k.clone()
    S.pa_paged_append(q2, k2, None, pos, None, None, None, rope_theta=1e4, q_out=q2, k_out=k2)
    assert torch.equal(q2, want_q) and torch.equal(k2, want_k)
    kp = torch.zeros((1, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    none, _, ws = S.pa_paged_append(None, k, v, None, i32(np.arange(9)), kp, vp)
    assert none is None and ok(S, ws) == 0
    assert torch.equal(kp[0, :9], k) and torch.equal(vp[0, :9], v) and (kp[0, 9:] == 0).all()


def test_append_skips_and_records_a_slot_out_of_range(S):
    k = randn((3, 2, 64), torch.float32, 1)
    kp = torch.zeros((1, 16, 2, 64), device="cuda")
    vp = torch.zeros_like(kp)
    _, _, ws = S.pa_paged_append(None, k, k, None, i32([2, 16, 2 ** 31 - 1]), kp, vp)
    assert ok(S, ws) == -1
    assert torch.equal(kp[0, 2], k[0]) and (kp[0, 3:] == 0).all()


# -------------------------------------------------------------------- prompt
PROMPTS = [[1], [2, 1, 3], [127], [128], [129, 1], [64, 65, 63], [257, 300, 1, 5], [31, 33, 1, 1, 1, 200, 640], [1025]]


def run_prompt(S, lens, hq, hkv, d, dtype, seed, pad=0, strided=False, want_lse=True):
    n = sum(lens)
    if strided:
        fused = randn((n + pad, hq + 2 * hkv + 1, d), dtype, seed)
        q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:hq + 2 * hkv]
    else:
        q, k, v = (randn((n + pad, h, d), dtype, seed + i) for i, h in enumerate((hq, hkv, hkv)))
    if pad:
        for t in (q, k, v):
            t[n:] = float("nan")
    o = torch.full((n + pad, hq, d), 99.0, dtype=dtype, device="cuda")
    lse = torch.full((n + pad, hq), 99.0, device="cuda") if want_lse else None
    cu = i32(np.concatenate([[0], np.cumsum(lens)]))
    o, lse, ws = S.pa_prompt_attend(q, k, v, cu, o=o, lse=lse, want_lse=want_lse)
    assert ok(S, ws) == 0
    assert (o[n:] == 99).all() and (lse is None or (lse[n:] == 99).all())
    at = 0
    qh, kh, vh = (t.double().cpu().numpy() for t in (q, k, v))
    for b, m in enumerate(lens):
        want = so.attend_rows(qh[at:at + m], kh[at:at + m], vh[at:at + m], 0)
        check_rows(dtype, o[at:at + m], None if lse is None else lse[at:at + m], want, max(m, 1), f"prompt {b} of {m}")
        at += m
    return q, k, v, o, lse


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("lens", PROMPTS, ids=lambda v: "-".join(map(str, v)))
def test_prompt_lengths(S, dtype, lens):
    run_prompt(S, lens, 8, 2, 128, DTYPES[dtype], seed=sum(lens), pad=3)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", HEADS)
def test_prompt_heads(S, dtype, d, hq, hkv):
    run_prompt(S, [150, 1, 77], hq, hkv, d, DTYPES[dtype], seed=hq + d, strided=True, want_lse=d == 64)


def test_prompt_empty_requests(S):
    run_prompt(S, [0, 5, 0, 0, 130, 0], 4, 2, 64, torch.bfloat16, 3)
    q, k, v = (torch.zeros((0, h, 64), dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2))
    o, lse, ws = S.pa_prompt_attend(q, k, v, i32([0]))
    assert o.shape == (0, 4, 64) and ok(S, ws) == 0
    o, lse, ws = S.pa_prompt_attend(q, k, v, i32([0, 0, 0]))
    assert ok(S, ws) == 0


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_prompt_many_short_requests(S, dtype):
    rng = np.random.default_rng(5)
    run_prompt(S, rng.integers(0, 5, 1500).tolist(), 4, 2, 64, DTYPES[dtype], 5)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_prompt_masked_values_add_nothing(S, dtype, bad):
    # a request padded behind its 100 tokens with non-finite K and V: rows
    # before them are as without; rows that see them are non-finite
    dt = DTYPES[dtype]
    q, k, v = (randn((330, h, 128), dt, 40 + i) for i, h in enumerate((8, 2, 2)))
    cu = i32([0, 300, 330])
    o0, lse0, _ = S.pa_prompt_attend(q, k, v, cu)
    for t, rows in ((v, slice(100, 104)), (k, slice(100, 104)), (v, slice(297, 300))):
        t2 = t.clone()
        t2[rows] = bad
        kk, vv = (t2, v) if t is k else (k, t2)
        o, lse, ws = S.pa_prompt_attend(q, kk, vv, cu)
        assert ok(S, ws) == 0
        clean = rows.start
        assert torch.equal(o[:clean], o0[:clean]) and torch.equal(lse[:clean], lse0[:clean])
        assert torch.equal(o[300:], o0[300:])
        if t is v:
            assert not torch.isfinite(o[clean:300]).any()
            assert torch.equal(lse, lse0)


def test_prompt_one_column_of_a_visible_infinity(S):
    # only the column that holds it, only rows that see it, with its sign
    for dt in DTYPES.values():
        q, k, v = (randn((200, h, 64), dt, 50 + i) for i, h in enumerate((4, 2, 2)))
        o0, _, _ = S.pa_prompt_attend(q, k, v, i32([0, 200]))
        v2 = v.clone()
        v2[130, 0, 7], v2[140, 0, 7], v2[150, 1, 9] = float("inf"), -float("inf"), float("nan")
        o, _, _ = S.pa_prompt_attend(q, k, v2, i32([0, 200]))
        assert (o[130:140, :2, 7] == float("inf")).all()
        assert torch.isnan(o[140:, :2, 7]).all() and torch.isnan(o[150:, 2:, 9]).all()
        keep = torch.ones_like(o, dtype=torch.bool)
        keep[130:, :2, 7] = False
        keep[150:, 2:, 9] = False
        assert torch.equal(o[keep], o0[keep])


def test_prompt_records_bad_offsets(S):
    q, k, v = (randn((64, h, 64), torch.bfloat16, 60 + i) for i, h in enumerate((4, 2, 2)))
    want, _, _ = S.pa_prompt_attend(q, k, v, i32([0, 20, 64]))
    for cu in ([0, 20, 65], [0, 20, 10], [-4, 20, 64]):
        o = torch.full_like(q, 99.0)
        o, _, ws = S.pa_prompt_attend(q, k, v, i32(cu), o=o)
        assert ok(S, ws) == -1, cu
        if cu[0] == 0:
            assert torch.equal(o[:20], want[:20]) and (o[20:] == 99).all()
        else:
            assert (o[:20] == 99).all() and torch.equal(o[20:], want[20:])


# --------------------------------------------------------------------- paged
PAGED = [
    ([1], [1]), ([1], [500]), ([1, 1, 1, 1, 1], [1, 127, 128, 129, 2000]), ([1] * 33, list(range(1, 34))),
    ([4, 1, 2], [4, 900, 77]), ([0, 1, 0, 3], [50, 60, 0, 3]), ([64], [3000]), ([65, 1, 200], [65, 4000, 1111]),
    ([300], [300]), ([129, 3, 1, 1], [1025, 3, 640, 1]), ([16, 17, 15], [256, 128, 15]),
]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("page", [16, 128])
@pytest.mark.parametrize("case", PAGED, ids=lambda c: "q" + "-".join(map(str, c[0][:6])))
def test_paged_lengths(S, dtype, page, case):
    c = paged_batch(*case, 8, 2, 128, page, DTYPES[dtype], seed=len(case[0]) + page, pad=2)
    o = torch.full_like(c["q"], 99.0)
    lse = torch.full(o.shape[:2], 99.0, device="cuda")
    o, lse, ws = S.pa_paged_attend(c["q"], c["cu_q"], c["kv_len"], c["table"], c["k_pages"], c["v_pages"], c["max_q"],
                                   o=o, lse=lse)
    assert ok(S, ws) == 0
    n = c["n"]
    assert (o[n:] == 99).all() and (lse[n:] == 99).all()
    check_paged(c, o[:n], lse[:n], "paged")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("case", [([1, 1, 1], [700, 1, 33]), ([2, 30, 1], [130, 300, 99])], ids=["decode", "chunk"])
def test_paged_heads(S, dtype, d, hq, hkv, case):
    page = 32 if d == 64 else 64
    c = paged_batch(*case, hq, hkv, d, page, DTYPES[dtype], seed=hq * d)
    o, lse, ws = S.pa_paged_attend(c["q"], c["cu_q"], c["kv_len"], c["table"], c["k_pages"], c["v_pages"], c["max_q"])
    assert ok(S, ws) == 0
    check_paged(c, o, lse, "paged")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("q_lens,kv_lens,hkv", [([64], [30000], 1), ([40, 1], [9000, 12000], 2), ([2], [70000], 1)])
def test_paged_keys_cut_into_many_pieces(S, dtype, q_lens, kv_lens, hkv):
    # few rows over long caches: more than 32 partial results per row
    c = paged_batch(q_lens, kv_lens, 4 * hkv, hkv, 64, 64, DTYPES[dtype], seed=8)
    o, lse, ws = S.pa_paged_attend(c["q"], c["cu_q"], c["kv_len"], c["table"], c["k_pages"], c["v_pages"], c["max_q"])
    assert ok(S, ws) == 0
    check_paged(c, o, lse, "many pieces")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("q_lens,kv_lens", [([3, 1, 5], [1, 0, 5]), ([40, 130], [3, 100]), ([1], [0])])
def test_paged_rows_that_see_nothing(S, dtype, q_lens, kv_lens):
    c = paged_batch(q_lens, kv_lens, 8, 2, 64, 16, DTYPES[dtype], seed=9)
    o, lse, ws = S.pa_paged_attend(c["q"], c["cu_q"], c["kv_len"], c["table"], c["k_pages"], c["v_pages"], c["max_q"])
    assert ok(S, ws) == 0
    check_paged(c, o, lse, "empty rows")
    assert (o[torch.isneginf(lse)] == 0).all() and torch.isneginf(lse).any()


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("q_len", [2, 5, 40])
def test_paged_masked_values_add_nothing(S, dtype, q_len):
    # the last new token's V is infinite: only its own row sees it
    c = paged_batch([q_len], [200], 4, 2, 64, 16, DTYPES[dtype], seed=3, poison=False)
    args = (c["q"], c["cu_q"], c["kv_len"], c["table"])
    o0, lse0, _ = S.pa_paged_attend(*args, c["k_pages"], c["v_pages"], q_len)
    v = c["v_pages"].clone()
    v[c["host_table"][0, 199 // 16], 199 % 16] = float("inf")
    o, lse, ws = S.pa_paged_attend(*args, c["k_pages"], v, q_len)
    assert ok(S, ws) == 0
    assert torch.equal(o[:-1], o0[:-1]) and torch.equal(lse, lse0)
    assert (o[-1] == float("inf")).all()


def test_paged_records_bad_lengths_and_pages(S):
    c = paged_batch([1, 1, 1], [40, 50, 60], 8, 2, 64, 16, torch.bfloat16, seed=4, poison=False)
    run = lambda kv, t, mq=1: S.pa_paged_attend(c["q"], c["cu_q"], kv, t, c["k_pages"], c["v_pages"], mq,
                                                o=torch.full_like(c["q"], 99.0))
    o0, _, ws = run(c["kv_len"], c["table"])
    assert ok(S, ws) == 0
    for kv in ([40, -1, 60], [40, c["table"].shape[1] * 16 + 1, 60]):
        o, _, ws = run(i32(kv), c["table"])
        assert ok(S, ws) == -1
        assert torch.equal(o[0], o0[0]) and torch.equal(o[2], o0[2]) and (o[1] == 99).all()
    for page in (-1, c["k_pages"].shape[0], 2 ** 31 - 1, -2 ** 31):
        t = c["table"].clone()
        t[1, 1] = page
        o, _, ws = run(c["kv_len"], t)
        assert ok(S, ws) == -1, page
        assert torch.equal(o[0], o0[0]) and torch.equal(o[2], o0[2])
    c = paged_batch([2, 1], [40, 50], 8, 2, 64, 16, torch.bfloat16, seed=4, poison=False)
    o, _, ws = S.pa_paged_attend(c["q"], c["cu_q"], c["kv_len"], c["table"], c["k_pages"], c["v_pages"], 1,
                                 o=torch.full_like(c["q"], 99.0))
    assert ok(S, ws) == -1 and (o[:2] == 99).all() and torch.isfinite(o[2]).all() and (o[2] != 99).any()


def test_paged_strided_rows_and_table(S):
    c = paged_batch([1, 70, 3], [90, 200, 3], 8, 2, 64, 32, torch.bfloat16, seed=6)
    args = lambda q, t: (q, c["cu_q"], c["kv_len"], t, c["k_pages"], c["v_pages"], c["max_q"])
    o0, lse0, _ = S.pa_paged_attend(*args(c["q"], c["table"]))
    fused = torch.full((c["q"].shape[0], 12, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    fused[:, 2:10] = c["q"]
    wide = torch.full((3, c["table"].shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    wide[:, :-5] = c["table"]
    o, lse, ws = S.pa_paged_attend(*args(fused[:, 2:10], wide[:, :-5]))
    assert ok(S, ws) == 0 and torch.equal(o, o0) and torch.equal(lse, lse0)


@pytest.mark.parametrize("page", [256, 1024, 32768])
def test_paged_large_pages(S, page):
    for case in (([1, 1, 2], [700, 1, 300]), ([90, 1], [700, 300])):
        c = paged_batch(*case, 8, 2, 64, page, torch.bfloat16, seed=page)
        o, lse, ws = S.pa_paged_attend(c["q"], c["cu_q"], c["kv_len"], c["table"], c["k_pages"], c["v_pages"], c["max_q"])
        assert ok(S, ws) == 0
        check_paged(c, o, lse, f"page {page}")


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_paged_the_most_requests(S, dtype):
    rng = np.random.default_rng(2)
    kv = rng.integers(0, 40, 8192)
    q = np.where(rng.random(8192) < 0.9, 1, 0)
    c = paged_batch(q.tolist(), kv.tolist(), 4, 2, 64, 16, DTYPES[dtype], seed=2)
    o, lse, ws = S.pa_paged_attend(c["q"], c["cu_q"], c["kv_len"], c["table"], c["k_pages"], c["v_pages"], 1)
    assert ok(S, ws) == 0
    check_paged(c, o, lse, "8192 requests")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("q_lens,kv_lens", [
    ([17] * 14 + [33] + [17] * 15, [40 + i for i in range(14)] + [3000] + [17 + 9 * i for i in range(15)]),
    ([20, 260, 1] * 11, [2500, 260, 1] + [30, 270, 60] * 10),
])
def test_paged_a_long_cache_beside_many_short_ones(S, dtype, q_lens, kv_lens):
    # more than three waves of row groups, and still the long one's keys are cut
    c = paged_batch(q_lens, kv_lens, 16, 16, 64, 16, DTYPES[dtype], seed=31)
    o, lse, ws = S.pa_paged_attend(c["q"], c["cu_q"], c["kv_len"], c["table"], c["k_pages"], c["v_pages"], c["max_q"])
    assert ok(S, ws) == 0
    check_paged(c, o, lse, "long beside short")


@pytest.mark.parametrize("bad", [0.0, float("inf"), float("nan")])
@pytest.mark.parametrize("q_lens,kv_lens", [
    ([70, 1, 2, 1], [900, 30, 2, 300]),          # the few tokens' keys are few: one kernel for all
    ([70, 1, 2, 1], [900, 30, 2, 1400]),         # a cache longer than the chunk's: the decode kernel
    ([2, 1, 40, 0, 1], [1, 0, 40, 9, 128]),      # rows and requests without a key
])
def test_paged_few_tokens_beside_a_chunk(S, q_lens, kv_lens, bad):
    c = paged_batch(q_lens, kv_lens, 8, 2, 128, 16, torch.bfloat16, seed=32)
    args = (c["cu_q"], c["kv_len"], c["table"])
    o, lse, ws = S.pa_paged_attend(c["q"], *args, c["k_pages"], c["v_pages"], c["max_q"])
    assert ok(S, ws) == 0
    check_paged(c, o, lse, "few tokens")
    # what the pages hold behind the last key changes nothing
    k, v = c["k_pages"].clone(), c["v_pages"].clone()
    for b, n in enumerate(kv_lens):
        for key in range(n, -(-n // 16) * 16):
            page = int(c["table"][b, key // 16])
            k[page, key % 16], v[page, key % 16] = bad, bad
    o1, lse1, ws = S.pa_paged_attend(c["q"], *args, k, v, c["max_q"])
    assert ok(S, ws) == 0 and torch.equal(o, o1) and torch.equal(lse, lse1)


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [300, 200]), ([4], [300]), ([70], [400]), ([200], [200])])
def test_a_bad_query_row_touches_no_other(S, dtype, bad, q_lens, kv_lens):
    c = paged_batch(q_lens, kv_lens, 8, 2, 64, 16, DTYPES[dtype], seed=21)
    args = (c["cu_q"], c["kv_len"], c["table"], c["k_pages"], c["v_pages"], c["max_q"])
    o0, lse0, _ = S.pa_paged_attend(c["q"], *args)
    q = c["q"].clone()
    q[c["n"] // 2, 3] = bad
    o, lse, ws = S.pa_paged_attend(q, *args)
    assert ok(S, ws) == 0
    keep = torch.ones(q.shape[:2], dtype=torch.bool, device="cuda")
    keep[c["n"] // 2, 3] = False
    assert torch.equal(o[keep], o0[keep]) and torch.equal(lse[keep], lse0[keep])
    assert torch.isnan(o[c["n"] // 2, 3]).all()


def test_scores_far_apart(S):
    # scores of hundreds: the running maximum moves from tile to tile, most
    # probabilities underflow, and nothing overflows
    for dt in DTYPES.values():
        for q_lens, kv_lens in (([1, 2], [900, 500]), ([130], [700])):
            c = paged_batch(q_lens, kv_lens, 4, 2, 64, 16, dt, seed=22)
            q = c["q"] * 40
            o, lse, ws = S.pa_paged_attend(q, c["cu_q"], c["kv_len"], c["table"], c["k_pages"], c["v_pages"], c["max_q"])
            assert ok(S, ws) == 0
            check_paged(dict(c, q=q), o, lse, "far apart")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,n", [(31, 700), (8001, 64), (201, 3)])
def test_offsets_that_count_rows_twice_stay_inside_the_workspace(S, dtype, B, n):
    # cu_q = 0, n, 0, n, ...: every other request has all the rows, together far
    # more than the call has; the rest falls and is recorded.  A second workspace
    # behind the first one is left as it was, and a good call in the same one is right.
    cu = torch.tensor([0, n] * ((B + 1) // 2), dtype=torch.int32, device="cuda")
    q, k, v = randn((n, 8, 64), DTYPES[dtype], 1), randn((n, 2, 64), DTYPES[dtype], 2), randn((n, 2, 64), DTYPES[dtype], 3)
    need = S._lib.pa_prompt_attend_workspace_size(B, n, 8, 2, 64, 1 if dtype == "bf16" else 0)
    whole = torch.full((need + 65536,), 93, dtype=torch.uint8, device="cuda")
    _, _, ws = S.pa_prompt_attend(q, k, v, cu, ws=whole[:need])
    assert ok(S, ws) == -1 and (whole[need:] == 93).all()
    kp, vp = randn((n // 16 + 1, 16, 2, 64), DTYPES[dtype], 4), randn((n // 16 + 1, 16, 2, 64), DTYPES[dtype], 5)
    table = torch.arange(n // 16 + 1, dtype=torch.int32, device="cuda").repeat(B, 1)
    kv = torch.full((B,), n, dtype=torch.int32, device="cuda")
    need = S._lib.pa_paged_attend_workspace_size(B, n, n, table.shape[1], 16, 8, 2, 64, 1 if dtype == "bf16" else 0)
    whole = torch.full((need + 65536,), 93, dtype=torch.uint8, device="cuda")
    _, _, ws = S.pa_paged_attend(q, cu, kv, table, kp, vp, n, ws=whole[:need])
    assert ok(S, ws) == -1 and (whole[need:] == 93).all()
    cu = torch.full((B + 1,), n, dtype=torch.int32, device="cuda")
    cu[0] = 0
    o, lse, ws = S.pa_paged_attend(q, cu, kv, table, kp, vp, n, ws=whole[:need])
    assert ok(S, ws) == 0 and (whole[need:] == 93).all()
    o1, lse1, _ = S.pa_paged_attend(q, cu[:2], kv[:1], table[:1], kp, vp, n)
    # each answer: P rounded (half a step of |v|) and o rounded (half a step of |o| <= |v|)
    tol = 4 * 2.0 ** -8 * float(vp.float().abs().max())
    assert (o.float() - o1.float()).abs().max() <= tol and (lse - lse1).abs().max() <= 1e-4


def test_empty_calls(S):
    t = torch.zeros((0, 4), dtype=torch.int32, device="cuda")
    none = i32(np.zeros(0))
    cu, kv, pos, slots, used, ws = S.pa_paged_schedule(none, none, t, none, 16, 3)
    assert ok(S, ws) == 0 and cu.tolist() == [0] and slots.tolist() == [-1] * 3 and pos.tolist() == [0] * 3
    assert used.tolist() == [0] and kv.numel() == 0
    k = torch.zeros((0, 2, 64), dtype=torch.bfloat16, device="cuda")
    kp = torch.zeros((1, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    q, ko, ws = S.pa_paged_append(torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda"), k, k, none, none, kp, kp,
                                  rope_theta=1e4, want_k=True)
    assert q.shape == (0, 4, 64) and ko.shape == (0, 2, 64) and ok(S, ws) == 0
    o, lse, ws = S.pa_paged_attend(q, i32([0, 0]), i32([5]), i32([[0]]), kp, kp, 1)
    assert o.shape == (0, 4, 64) and ok(S, ws) == 0
    # a cache without pages: every key reads as zero, and is recorded
    q = torch.ones((1, 4, 64), dtype=torch.bfloat16, device="cuda")
    no = torch.zeros((0, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    for m in (1, 5):
        q = torch.ones((m, 4, 64), dtype=torch.bfloat16, device="cuda")
        o, lse, ws = S.pa_paged_attend(q, i32([0, m]), i32([m]), i32([[0]]), no, no, m)
        assert ok(S, ws) == -1 and (o == 0).all()


def test_calls_on_two_streams_and_repeated(S):
    # the same inputs give the same bits, on any stream, with a fresh or a used workspace
    c = paged_batch([1, 40, 1], [3000, 900, 20], 8, 2, 128, 16, torch.bfloat16, seed=7)
    args = (c["q"], c["cu_q"], c["kv_len"], c["table"], c["k_pages"], c["v_pages"], c["max_q"])
    o0, lse0, ws = S.pa_paged_attend(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(4):
        with torch.cuda.stream(side):
            o1, lse1, _ = S.pa_paged_attend(*args)
        o2, lse2, _ = S.pa_paged_attend(*args, ws=ws)
        torch.cuda.synchronize()
        for o, lse in ((o1, lse1), (o2, lse2)):
            assert torch.equal(o, o0) and torch.equal(lse, lse0)


def test_calls_from_several_threads(S):
    c = paged_batch([1, 64, 5], [30, 200, 90], 8, 2, 64, 16, torch.bfloat16, seed=33)
    args = (c["q"], c["cu_q"], c["kv_len"], c["table"], c["k_pages"], c["v_pages"], c["max_q"])
    want, want_lse, _ = S.pa_paged_attend(*args)
    torch.cuda.synchronize()
    wrong, done = [], []

    def work(i):
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            got = [S.pa_paged_attend(*args)[:2] for _ in range(20)]
            side.synchronize()
        wrong.extend(i for o, lse in got if not (torch.equal(o, want) and torch.equal(lse, want_lse)))
        done.append(i)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong and len(done) == 4


FIRST_CALL = """
import torch
from long_context_blockwise_max_b200 import serving as S
q = torch.randn(70, 8, 64, device="cuda").bfloat16()
k, v = (torch.randn(40, 16, 2, 64, device="cuda").bfloat16() for _ in range(2))
cu, kv = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([0, 1, 65, 70], [30, 200, 90]))
t = torch.arange(39, dtype=torch.int32, device="cuda").view(3, 13)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    o, lse, ws = S.pa_paged_attend(q, cu, kv, t, k, v, 64)
g.replay()
o1, lse1, _ = S.pa_paged_attend(q, cu, kv, t, k, v, 64)
assert torch.equal(o, o1) and torch.equal(lse, lse1)
print("captured")
"""


def test_a_process_may_capture_its_first_call():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    got = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert got.returncode == 0 and "captured" in got.stdout, got.stderr[-2000:]


def test_captured_step_follows_its_inputs(S):
    # one captured graph of a whole step, replayed with other lengths and
    # another graph sharing its workspace replayed in between
    hq, hkv, d, page, B, pages = 8, 2, 64, 16, 4, 64
    dt = torch.bfloat16
    q_len, kv_len = i32([1, 1, 1, 1]), i32([5, 100, 0, 33])
    table = torch.zeros((B, 16), dtype=torch.int32, device="cuda")
    free = torch.arange(pages, dtype=torch.int32, device="cuda")
    kp = torch.zeros((pages, page, hkv, d), dtype=dt, device="cuda")
    vp = torch.zeros_like(kp)
    x = randn((6, hq + 2 * hkv, d), dt, 8)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")

    def step():
        cu, kv, pos, slots, used, w0 = S.pa_paged_schedule(q_len, kv_len, table, free, page, 6)
        q, _, w1 = S.pa_paged_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos, slots, kp, vp, rope_theta=1e4)
        o, lse, _ = S.pa_paged_attend(q, cu, kv, table, kp, vp, 3, ws=ws)
        return cu, kv, slots, q, o, lse

    step()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = step()
        graphs.append((g, out))
    for lens, ctx in (([1, 1, 1, 1], [5, 100, 0, 33]), ([3, 0, 2, 1], [0, 7, 31, 200]), ([1, 2, 0, 1], [15, 16, 17, 18])):
        rng = np.random.default_rng(sum(ctx))
        tab = np.zeros((B, 16), dtype=np.int64)
        order = rng.permutation(pages)
        at = 0
        for b, c in enumerate(ctx):
            h = -(-c // page)
            tab[b, :h] = order[at:at + h]
            at += h
        kp.copy_(randn(kp.shape, dt, 11 + sum(ctx)))
        vp.copy_(randn(vp.shape, dt, 12 + sum(ctx)))
        q_len.copy_(i32(lens))
        kv_len.copy_(i32(ctx))
        table.copy_(i32(tab))
        f = np.full(pages, 2 ** 30, dtype=np.int64)
        f[:pages - at] = order[at:]
        free.copy_(i32(f))
        for g, out in graphs:
            g.replay()
        torch.cuda.synchronize()
        for g, (cu, kv, slots, q, o, lse) in graphs:
            n = sum(lens)
            c = dict(q=q, k_pages=kp, v_pages=vp, host_table=table.cpu().numpy(), q_lens=lens,
                     kv_lens=[a + b for a, b in zip(lens, ctx)])
            check_paged(c, o[:n], lse[:n], "captured")


def test_long_offsets_pass_32_bits(S):
    # a cache of more than 2^32 elements, its last pages in use
    hq, hkv, d, page = 16, 8, 128, 128
    n_pages = 2 ** 32 // (page * hkv * d) + 40
    kp = torch.zeros((n_pages, page, hkv, d), dtype=torch.bfloat16, device="cuda")
    vp = torch.zeros_like(kp)
    assert kp.numel() > 2 ** 32
    for q_lens, kv_lens in (([1, 1], [300, 1000]), ([200], [1000])):
        table = np.zeros((len(q_lens), 9), dtype=np.int64)
        for b, kv in enumerate(kv_lens):
            table[b, :8] = n_pages - 1 - 8 * b - np.arange(8)
        last = n_pages - 40
        kp[last:], vp[last:] = randn((40, page, hkv, d), torch.bfloat16, 1), randn((40, page, hkv, d), torch.bfloat16, 2)
        q = randn((sum(q_lens), hq, d), torch.bfloat16, 3)
        cu = np.concatenate([[0], np.cumsum(q_lens)])
        o, lse, ws = S.pa_paged_attend(q, i32(cu), i32(kv_lens), i32(table), kp, vp, max(q_lens))
        assert ok(S, ws) == 0
        c = dict(q=q, k_pages=kp[last:], v_pages=vp[last:], host_table=table - last, q_lens=q_lens, kv_lens=kv_lens)
        check_paged(c, o, lse, "long cache")
    # and the append to them
    k = randn((2, hkv, d), torch.bfloat16, 4)
    slots = [n_pages * page - 1, n_pages * page - 130]
    _, _, ws = S.pa_paged_append(None, k, k, None, i32(slots), kp, vp)
    assert ok(S, ws) == 0
    assert torch.equal(kp.view(-1, hkv, d)[slots], k) and torch.equal(vp.view(-1, hkv, d)[slots], k)


# ------------------------------------------------------- together, in earnest
@pytest.mark.parametrize("dtype", list(DTYPES))
def test_prompts_then_chunks_then_tokens(S, dtype):
    """Three requests: prompts through the packed kernel with their K and V
    appended, then a chunk each, then single tokens; every output is the
    row of causal attention over the request's whole sequence."""
    dt = DTYPES[dtype]
    hq, hkv, d, page, theta, B = 8, 2, 64, 16, 1e4, 3
    steps = [[70, 1, 33], [5, 64, 0], [1, 1, 1], [1, 1, 1]]
    pages = 40
    table = torch.full((B, 12), -1, dtype=torch.int32, device="cuda")
    pool = np.random.default_rng(1).permutation(pages)
    kp = torch.full((pages, page, hkv, d), float("nan"), dtype=dt, device="cuda")
    vp = kp.clone()
    kv = i32([0, 0, 0])
    taken = 0
    seen = [dict(q=[], k=[], v=[]) for _ in range(B)]
    for it, lens in enumerate(steps):
        n = sum(lens)
        x = randn((n, hq + 2 * hkv, d), dt, 100 + it)
        cu, kv, pos, slots, used, ws = S.pa_paged_schedule(i32(lens), kv, table, i32(pool[taken:]), page, n)
        assert ok(S, ws) == 0
        taken += int(used)
        q, k, ws = S.pa_paged_append(x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:], pos, slots, kp, vp,
                                     rope_theta=theta, want_k=True)
        assert ok(S, ws) == 0
        if it == 0:
            o, lse, ws = S.pa_prompt_attend(q, k, x[:, hq + hkv:], cu)
            o2, lse2, ws2 = S.pa_paged_attend(q, cu, kv, table, kp, vp, max(lens))
            assert ok(S, ws2) == 0
        else:
            o, lse, ws = S.pa_paged_attend(q, cu, kv, table, kp, vp, max(lens))
        assert ok(S, ws) == 0
        at = 0
        for b, m in enumerate(lens):
            before = sum(len(t) for t in seen[b]["k"])
            rows = slice(at, at + m)
            seen[b]["k"].append(k[rows].double().cpu().numpy())
            seen[b]["v"].append(x[rows, hq + hkv:].double().cpu().numpy())
            want = so.attend_rows(q[rows].double().cpu().numpy(), np.concatenate(seen[b]["k"]),
                                  np.concatenate(seen[b]["v"]), before)
            check_rows(dt, o[rows], lse[rows], want, before + max(m, 1), f"step {it}, request {b}")
            if it == 0:
                check_rows(dt, o2[rows], lse2[rows], want, max(m, 1), f"paged prompt {b}")
            at += m
    assert kv.tolist() == [sum(s[b] for s in steps) for b in range(B)]


def test_phase1_and_phase2_agree_with_the_pages(S):
    """Phase 1's retained cache is a paged cache in place: a paged query over it
    is Phase 2, and one Star host is a packed prompt."""
    from long_context_blockwise_max_b200 import pulsar as P
    L, hq, hkv, d, theta = 512, 8, 2, 128, 1e4
    q, k, v = (randn((L, h, d), torch.bfloat16, 30 + i) for i, h in enumerate((hq, hkv, hkv)))
    o1, lse1, k_ret, v_ret, _, ws = P.star_phase1_encode(q, k, v, theta, L)
    assert P.pa_workspace_status(ws) == 0
    pos = torch.arange(L, dtype=torch.int32, device="cuda")
    qr, kr, _ = S.pa_paged_append(q, k, None, pos, None, None, None, rope_theta=theta, want_k=True)
    o, lse, ws = S.pa_prompt_attend(qr, kr, v, i32([0, L]))
    assert ok(S, ws) == 0
    # both round the same rotation once (angles off by less than 2^-20 of |x1| + |x2|), so they are at most
    # two half steps apart: where it lies by a border between two bf16 values, neighbours
    x = k.float().abs()
    size = torch.cat([x[..., :d // 2] + x[..., d // 2:]] * 2, -1)
    step = half_step(torch.bfloat16)
    assert ((kr.float() - k_ret.float()).abs() <= 2 * (step * k_ret.float().abs() * (1 + step) + 2.0 ** -19 * size)).all()
    # Phase 1 keeps rotated Q and K in fp16 (2^-11 each), here they are rounded to bf16 (2^-8 each): scores are
    # ds = (2^-7 + 2^-10) * raw apart (1 % for the products), so probabilities by a factor within exp(2 ds)
    ref, _, mag, raw = so.attend_rows(*(t.double().cpu().numpy() for t in (qr, kr, v)), 0)
    ds = 1.01 * (2.0 ** -7 + 2.0 ** -10) * raw
    apart = np.abs(o.double().cpu().numpy() - o1.double().cpu().numpy())
    assert (apart <= (np.expm1(2 * ds) + 4 * step) * mag * (1 + step)).all()
    query = randn((1, 3, hq, d), torch.bfloat16, 40)
    want, wlse, _, _, ws = P.star_phase2_attend(query, k_ret[None], v_ret[None], 4)
    pages = k_ret.view(-1, 64, hkv, d), v_ret.view(-1, 64, hkv, d)
    table = torch.arange(L // 64, dtype=torch.int32, device="cuda")
    # three requests of one token share the pages: no causal limit among them, as in Phase 2
    got, glse, ws = S.pa_paged_attend(query[0], i32([0, 1, 2, 3]), i32([L] * 3), table.repeat(3, 1), *pages, 1)
    assert ok(S, ws) == 0
    ref = [so.attend_rows(query[0, i:i + 1].double().cpu().numpy(), k_ret.double().cpu().numpy(),
                          v_ret.double().cpu().numpy(), L - 1) for i in range(3)]
    for i in range(3):
        check_rows(torch.bfloat16, got[i:i + 1], glse[i:i + 1], ref[i], L, "shared pages")
    assert (glse - wlse[0]).abs().max() <= 1e-3 and (got.float() - want[0].float()).abs().max() <= 2e-2


def test_outputs_stay_inside_their_buffers(S):
    # every output as a view into a buffer with sentinel rows on both sides
    c = paged_batch([1, 37, 1, 200], [500, 37, 9, 300], 28, 4, 64, 16, torch.bfloat16, seed=12)
    n, hq, d = c["q"].shape
    for run in ("paged", "decode", "prompt"):
        big_o = torch.full((n + 64, hq, d), 99.0, dtype=torch.bfloat16, device="cuda")
        big_l = torch.full((n + 64, hq), 99.0, device="cuda")
        if run == "prompt":
            k, v = randn((n, 4, d), torch.bfloat16, 1), randn((n, 4, d), torch.bfloat16, 2)
            rows = n
            S.pa_prompt_attend(c["q"], k, v, c["cu_q"], o=big_o[32:32 + n], lse=big_l[32:32 + n])
        elif run == "paged":
            rows = n
            S.pa_paged_attend(c["q"], c["cu_q"], c["kv_len"], c["table"], c["k_pages"], c["v_pages"], 200,
                              o=big_o[32:32 + n], lse=big_l[32:32 + n])
        else:
            rows = 2
            S.pa_paged_attend(c["q"], i32([0, 1, 1, 1, 2]), c["kv_len"], c["table"], c["k_pages"], c["v_pages"], 1,
                              o=big_o[32:32 + n], lse=big_l[32:32 + n])
        torch.cuda.synchronize()
        assert (big_o[:32] == 99).all() and (big_o[32 + rows:] == 99).all()
        assert (big_l[:32] == 99).all() and (big_l[32 + rows:] == 99).all()
        assert (big_l[32:32 + rows] != 99).all()


@pytest.mark.parametrize("case", [([1, 1], [700, 90]), ([40, 150], [300, 150])], ids=["decode", "tiles"])
def test_stalled_barrier_times_out_and_context_survives(S, case):
    import time
    c = paged_batch(*case, 8, 2, 128, 16, torch.bfloat16, seed=15, poison=False)
    args = (c["q"], c["cu_q"], c["kv_len"], c["table"], c["k_pages"], c["v_pages"], c["max_q"])
    t0 = time.time()
    assert ok(S, S.pa_testing_paged_stall(*args, wait_limit_us=20000)) == -5     # PA_ERR_TIMEOUT
    assert time.time() - t0 < 30.0
    o, lse, ws = S.pa_paged_attend(*args)
    assert ok(S, ws) == 0
    check_paged(c, o, lse, "after the stall")
