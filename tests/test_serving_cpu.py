"""Serving operators without a GPU: the header's symbols, the host-side checks
of the C ABI and of the binding, and the oracle they are tested against."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from long_context_blockwise_max_b200 import build
from oracle import serving_oracle as so

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def S():
    build.build()
    from long_context_blockwise_max_b200 import serving
    return serving


def test_library_exports_the_serving_header(S):
    src = open(os.path.join(ROOT, "include", "pulsar_serving.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    names = sorted(set(re.findall(r"^\s*(?:int|size_t)\s+(\w+)\s*\(", src, flags=re.M)))
    assert sorted(S.ABI_SYMBOLS) == names
    so_ = ctypes.CDLL(S.pulsar.LIB_PATH)
    for n in names:
        assert hasattr(so_, n), n
    assert S.pulsar.status_string(-7) == "page pool or page table too small"


def test_workspace_sizes(S):
    assert S.pa_prompt_attend_workspace_size(4, 1000, 32, 8, 128, 1) > 256
    assert S.pa_prompt_attend_workspace_size(4, 1000, 32, 8, 96, 1) == 0
    assert S.pa_prompt_attend_workspace_size(4, 1000, 65, 1, 128, 1) == 0
    assert S.pa_prompt_attend_workspace_size(8193, 10000, 32, 8, 128, 1) == 0
    assert S.pa_prompt_attend_workspace_size(4, 2 ** 31, 32, 8, 128, 1) == 0
    assert S.pa_paged_attend_workspace_size(4, 100, 1, 64, 16, 32, 8, 128, 1) > 256
    assert S.pa_paged_attend_workspace_size(4, 100, 1, 64, 24, 32, 8, 128, 1) == 0
    assert S.pa_paged_attend_workspace_size(4, 100, 0, 64, 16, 32, 8, 128, 1) == 0
    assert S.pa_paged_attend_workspace_size(4, 100, 1, 0, 16, 32, 8, 128, 1) == 0
    # bounded by what fits one launch, whatever the cache's length
    assert S.pa_paged_attend_workspace_size(16, 16, 1, 8192, 128, 32, 8, 128, 1) < 1 << 26


WS, X = ctypes.c_void_p(256), ctypes.c_void_p(4096)   # never dereferenced: validation fails first


def test_schedule_validation(S):
    f = S.pulsar._lib.pa_paged_schedule
    def call(B=4, stride=8, width=8, n_free=3, page=16, n=10, table=X, cu=X, pos=X, free=X, ws=WS, wsb=256):
        return f(X, X, B, table, stride, width, free, n_free, page, n, cu, X, pos, X, X, ws, wsb, None)
    assert call(B=-1) == -1 and call(B=8193) == -2
    assert call(n=-1) == -1 and call(n=2 ** 31) == -2
    assert call(stride=7) == -1 and call(width=0) == -1 and call(page=0) == -1
    for page in (8, 24, 65536):
        assert call(page=page) == -2
    assert call(width=2 ** 27, stride=2 ** 27) == -2
    assert call(n_free=-1) == -1 and call(free=None) == -1
    assert call(table=None) == -1 and call(cu=None) == -1 and call(pos=None) == -1
    assert call(ws=None) == -3 and call(wsb=255) == -3 and call(ws=ctypes.c_void_p(128)) == -3


def test_append_validation(S):
    f = S.pulsar._lib.pa_paged_append
    def call(q=X, k=X, v=X, dt=1, N=4, ldq=1024, ldk=256, ldv=256, hq=8, hkv=2, d=128, theta=1e4, pos=X, slots=X, kp=X,
             vp=X, n_slots=64, qo=X, ko=None, ws=WS, wsb=256):
        return f(q, k, v, dt, N, ldq, ldk, ldv, hq, hkv, d, theta, pos, slots, kp, vp, n_slots, qo, ko, ws, wsb, None)
    assert call(d=96) == -2 and call(dt=2) == -2 and call(hq=7) == -1 and call(hkv=0) == -1
    assert call(hq=130, hkv=2) == -2
    assert call(theta=-1.0) == -1 and call(theta=float("nan")) == -1 and call(theta=float("inf")) == -1
    assert call(ldq=1016) == -1 and call(ldk=255) == -1 and call(ldv=257) == -2
    assert call(slots=None) == -1 and call(vp=None) == -1 and call(v=None) == -1 and call(pos=None) == -1
    assert call(qo=None) == -1 and call(q=None) == -1
    assert call(n_slots=-1) == -1 and call(n_slots=2 ** 31) == -1
    assert call(k=ctypes.c_void_p(4104)) == -2 and call(ko=ctypes.c_void_p(4104)) == -2
    assert call(N=-1) == -1 and call(wsb=100) == -3


def test_attend_validation(S):
    lib = S.pulsar._lib
    def prompt(q=X, dt=1, N=64, ldq=1024, ldk=256, ldv=256, cu=X, B=2, hq=8, hkv=2, d=128, o=X, ws=WS, wsb=1 << 30):
        return lib.pa_prompt_attend(q, X, X, dt, N, ldq, ldk, ldv, cu, B, hq, hkv, d, o, None, ws, wsb, None)
    assert prompt(d=32) == -2 and prompt(dt=7) == -2 and prompt(hq=9) == -1 and prompt(hq=65, hkv=1) == -2
    assert prompt(B=-1) == -1 and prompt(N=-1) == -1 and prompt(B=9000) == -2
    assert prompt(cu=None) == -1 and prompt(q=None) == -1 and prompt(o=None) == -1
    assert prompt(ldq=1020) == -1 and prompt(ldk=257) == -2
    assert prompt(q=ctypes.c_void_p(4098)) == -2 and prompt(o=ctypes.c_void_p(4104)) == -2
    assert prompt(wsb=300) == -3 and prompt(ws=ctypes.c_void_p(300)) == -3

    def paged(N=4, ldq=1024, max_q=1, stride=16, width=16, page=16, n_pages=9, hq=8, hkv=2, d=128, kv=X, table=X, kp=X,
              wsb=1 << 30, B=4):
        return lib.pa_paged_attend(X, 1, N, ldq, X, kv, B, max_q, table, stride, width, page, kp, X, n_pages, hq, hkv, d,
                                   X, None, WS, wsb, None)
    assert paged(max_q=0) == -1 and paged(stride=15) == -1 and paged(width=0) == -1
    assert paged(page=48) == -2 and paged(page=8) == -2
    assert paged(n_pages=-1) == -1 and paged(n_pages=2 ** 28) == -2
    assert paged(kv=None) == -1 and paged(table=None) == -1 and paged(kp=None) == -1
    assert paged(kp=ctypes.c_void_p(4100)) == -2 and paged(ldq=1016) == -1 and paged(d=256) == -2
    assert paged(wsb=1000) == -3


def test_binding_refuses_mismatched_tensors(S, monkeypatch):
    # CPU tensors with the device check stubbed out: these stop before the library
    with pytest.raises(ValueError, match="CUDA"):
        S.pa_prompt_attend(*(torch.zeros((4, 2, 64)),) * 3, torch.zeros(2, dtype=torch.int32))
    monkeypatch.setattr(S, "_on", lambda *ts: None)
    i32, bf = torch.int32, torch.bfloat16
    q, k = torch.zeros((10, 8, 64), dtype=bf), torch.zeros((10, 2, 64), dtype=bf)
    cu, kv = torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32)
    table, kp = torch.zeros((2, 4), dtype=i32), torch.zeros((6, 16, 2, 64), dtype=bf)

    def bad(match, f, *a, **kw):
        with pytest.raises(ValueError, match=match):
            f(*a, **kw)
    pr, pg, ap, sc = S.pa_prompt_attend, S.pa_paged_attend, S.pa_paged_append, S.pa_paged_schedule
    bad("q:", pr, q[0], k, k, cu)
    bad("heads of a token", pr, q.transpose(1, 2).contiguous().transpose(1, 2), k, k, cu)
    bad("overlap", pr, q[:1].expand(10, 8, 64), k, k, cu)
    bad("k:", pr, q, k[:9], k[:9], cu)
    bad("v:", pr, q, k, k[:, :1], cu)
    bad("k: head dimension", pr, q, torch.zeros((10, 2, 128), dtype=bf), k, cu)
    bad("cu_q", pr, q, k, k, cu.long())
    bad("o:", pr, q, k, k, cu, o=torch.zeros((10, 8, 64)))
    bad("o:", pr, q, k, k, cu, o=q[:9].clone())
    bad("lse:", pr, q, k, k, cu, lse=torch.zeros((10, 7)))
    bad("must not be q", pr, q, k, k, cu, o=q)
    bad("kv_len", pg, q, cu, kv[:1], table, kp, kp, 1)
    bad("block_table", pg, q, cu, kv, table[:1], kp, kp, 1)
    bad("block_table", pg, q, cu, kv, table.long(), kp, kp, 1)
    bad("block_table", pg, q, cu, kv, table.t().contiguous().t(), kp, kp, 1)
    bad("block_table: rows overlap", pg, q, cu, kv, table[:1].expand(2, 4), kp, kp, 1)
    bad("v_pages", pg, q, cu, kv, table, kp, kp[:5], 1)
    bad("k_pages", pg, q, cu, kv, table, kp.float(), kp.float(), 1)
    bad("k_pages", pg, q, cu, kv, table, kp[:, :, :, :32].contiguous(), kp[:, :, :, :32].contiguous(), 1)
    bad("contiguous", pg, q, cu, kv, table, kp[:, ::2], kp[:, ::2], 1)
    pos = torch.zeros(10, dtype=i32)
    bad("together", ap, q, k, k, pos, pos, kp, None)
    bad("positions", ap, q, k, k, None, pos, kp, kp, rope_theta=1e4)
    bad("slots", ap, q, k, k, pos, pos[:9], kp, kp)
    bad("v_new", ap, q, k, None, pos, pos, kp, kp)
    bad("v_new", ap, q, k, k[:9], pos, pos, kp, kp)
    bad("kv heads", ap, q, k, k, pos, pos, torch.zeros((6, 16, 1, 64), dtype=bf), torch.zeros((6, 16, 1, 64), dtype=bf))
    bad("q:", ap, q.float(), k, k, pos, pos, kp, kp)
    bad("q_out", ap, None, k, k, pos, pos, kp, kp, q_out=q)
    fused = torch.zeros((10, 12, 64), dtype=bf)
    bad("in place", ap, fused[:, :8], k, k, pos, pos, kp, kp, q_out=fused.view(-1)[:10 * 8 * 64])
    bad("q_len", sc, kv.long(), kv, table, pos, 16, 4)
    bad("kv_len_out", sc, kv, kv, table, pos, 16, 4, kv_len_out=kv)
    bad("slots", sc, kv, kv, table, pos, 16, 4, slots=pos[:3])
    bad("cu_q", sc, kv, kv, table, pos, 16, 4, cu_q=pos[:2])


def test_binding_refuses_outputs_over_inputs(S, monkeypatch):
    monkeypatch.setattr(S, "_on", lambda *ts: None)
    i32, bf = torch.int32, torch.bfloat16
    flat = torch.zeros(40 * 8 * 64, dtype=bf)
    q, k, v = flat[:10 * 8 * 64].view(10, 8, 64), torch.zeros((10, 2, 64), dtype=bf), torch.zeros((10, 2, 64), dtype=bf)
    late = flat[512:512 + 10 * 8 * 64]          # q, one token later
    cu, kv, pos = torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(10, dtype=i32)
    table, kp = torch.zeros((2, 4), dtype=i32), torch.zeros((6, 16, 2, 64), dtype=bf)
    vp = torch.zeros_like(kp)
    ints = torch.zeros(40, dtype=i32)

    def bad(match, f, *a, **kw):
        with pytest.raises(ValueError, match=match):
            f(*a, **kw)
    pr, pg, ap, sc = S.pa_prompt_attend, S.pa_paged_attend, S.pa_paged_append, S.pa_paged_schedule
    bad("o: overlaps q", pr, q, k, v, cu, o=late)
    bad("o: overlaps lse", pr, q, k, v, cu, o=flat[10240:15360], lse=flat[10240:].view(torch.float32))
    bad("o: overlaps v_pages", pg, q, cu, kv, table, kp, vp, 1, o=vp.view(-1)[:5120])
    bad("q_out: overlaps q", ap, q, k, v, pos, pos.clone(), kp, vp, q_out=late)
    bad("q_out: overlaps k_pages", ap, q, k, v, pos, pos.clone(), kp, vp, q_out=kp.view(-1)[64:])
    bad("k_out: overlaps v_new", ap, q, k, v, pos, pos.clone(), kp, vp, k_out=v)
    bad("k_pages: overlaps v_pages", ap, q, k, v, pos, pos.clone(), kp, kp)
    bad("v_pages: overlaps k_new", ap, q, vp.view(-1, 2, 64)[3:13], v, pos, pos.clone(), kp, vp)
    bad("kv_len_out: overlaps kv_len", sc, ints[20:22], ints[:2], table, pos, 16, 4, kv_len_out=ints[1:3])
    bad("positions: overlaps slots", sc, kv, kv, table, pos, 16, 4, positions=ints[:4], slots=ints[3:8])
    bad("block_table: overlaps free_pages", sc, kv, kv, table, table.view(-1), 16, 4)


def test_oracle_attention_against_library_attention():
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn((n, h, 32), generator=g, dtype=torch.float64) for n, h in ((7, 6), (19, 2), (19, 2)))
    o, lse, mag, raw = so.attend_rows(q, k, v, 12)
    mask = torch.arange(19) <= 12 + torch.arange(7)[:, None]
    want = torch.nn.functional.scaled_dot_product_attention(
        q.transpose(0, 1), k.transpose(0, 1), v.transpose(0, 1), attn_mask=mask, enable_gqa=True).transpose(0, 1)
    assert np.allclose(o, want.numpy(), atol=1e-12)
    s = torch.einsum("nhd,thd->hnt", q, k.repeat_interleave(3, 1)) / 32 ** 0.5
    s = s.masked_fill(~mask, -float("inf"))
    assert np.allclose(lse, torch.logsumexp(s, -1).T.numpy(), atol=1e-12)
    assert (mag >= np.abs(o)).all() and raw >= np.abs(s[torch.isfinite(s)].numpy()).max()
    o, lse, _, _ = so.attend_rows(q[:3], k[:1], v[:1], -2)
    assert np.isneginf(lse[:2]).all() and (o[:2] == 0).all() and np.allclose(o[2], v[:1].numpy().repeat(3, 1)[0])


def test_oracle_schedule_by_hand():
    # page 16: request 0 has 15 tokens in page 4, its 2 new ones end in a new
    # page; request 1 is new with 17 tokens (two pages); request 2 is idle
    cu, kv, pos, slots, used, table, refused = so.schedule_step(
        [2, 17, 0], [15, 0, 3], [[4, -1], [-1, -1], [8, -1]], [9, 2, 5, 1], 16, 20)
    assert cu.tolist() == [0, 2, 19, 19] and kv.tolist() == [17, 17, 3] and used == 3 and not refused
    assert table.tolist() == [[4, 9], [2, 5], [8, -1]]
    assert pos.tolist() == [15, 16] + list(range(17)) + [0]
    assert slots.tolist() == [79, 144] + list(range(32, 48)) + [80] + [-1]


def test_oracle_rope_matches_the_rotation_formula():
    x = np.random.default_rng(1).standard_normal((3, 2, 8))
    pos, theta = np.array([0, 5, 1000]), 1e4
    y = so.rope(x, pos, theta)
    for t in range(3):
        for m in range(4):
            a = pos[t] * theta ** (-2 * m / 8)
            assert np.allclose(y[t, :, m], x[t, :, m] * np.cos(a) - x[t, :, m + 4] * np.sin(a))
            assert np.allclose(y[t, :, m + 4], x[t, :, m + 4] * np.cos(a) + x[t, :, m] * np.sin(a))
    assert np.array_equal(so.rope(x, pos, 0), x)
