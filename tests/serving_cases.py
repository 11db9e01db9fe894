"""Inputs and tolerances of the serving operators' tests."""
import numpy as np
import torch

from oracle import serving_oracle as so

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def half_step(dtype):
    """Relative error of one rounding to ``dtype``."""
    return torch.finfo(dtype).eps / 2


def bounds(dtype, o, lse, mag, raw, n_keys, d):
    """(bound on |o error| per element, bound on |lse error|).

    A score's fp32 products and sums are off by at most d * 2^-24 * raw (raw =
    max sum |q_m k_m| / sqrt(d)), its scaling and the subtraction of the
    maximum by a few 2^-24 of the score, |score| <= raw: ds = (d + 8) * 2^-24 *
    raw.  exp and log then err by a few 2^-23 and the sums over n keys by
    n * 2^-24, so a probability is off by 2 ds + (n + 16) * 2^-23 relatively,
    which acts on mag = sum p |v|.  bf16 adds one rounding of the
    probabilities (on mag) and one of o."""
    ds = (d + 8) * 2.0 ** -24 * raw
    rel = 2 * ds + (n_keys + 16) * 2.0 ** -23
    if dtype == torch.bfloat16:
        rel += half_step(dtype)
    b_o = rel * mag + half_step(dtype) * (np.abs(o) + rel * mag) + 1e-30
    b_lse = ds + (n_keys + 16) * 2.0 ** -23 + 2.0 ** -22 * np.where(np.isfinite(lse), np.abs(lse), 0)
    return b_o, b_lse


def check_rows(dtype, got_o, got_lse, want, n_keys, what):
    o, lse, mag, raw = want
    b_o, b_lse = bounds(dtype, o, lse, mag, raw, n_keys, o.shape[-1])
    go = got_o.double().cpu().numpy()
    assert np.isfinite(go).all(), f"{what}: o is not finite"
    over = np.abs(go - o) - b_o
    assert (over <= 0).all(), f"{what}: o off by {np.abs(go - o).max():.3e}, {over.max():.3e} over its bound"
    if got_lse is not None:
        gl = got_lse.double().cpu().numpy()
        empty = np.isneginf(lse)
        assert np.array_equal(np.isneginf(gl), empty), f"{what}: empty rows"
        err = np.where(empty, 0, np.abs(np.where(empty, 0, gl) - np.where(empty, 0, lse)))
        assert (err <= b_lse).all(), f"{what}: lse off by {err.max():.3e}"


def randn(shape, dtype, seed, device="cuda"):
    gen = torch.Generator(device="cpu").manual_seed(seed)
    return torch.randn(shape, generator=gen).to(dtype).to(device)


def paged_batch(q_lens, kv_lens, hq, hkv, d, page, dtype, seed, device="cuda", poison=True, pad=0):
    """A packed batch over shuffled pages.  With ``poison`` every cache slot
    that holds no key is NaN, unused table entries are out of range, and the
    padding rows of q are NaN.  Returns a dict of tensors and host copies."""
    rng = np.random.default_rng(seed)
    held = [-(-kv // page) for kv in kv_lens]
    n_pages = max(1, sum(held)) + 3
    order = rng.permutation(n_pages)
    width = max(held + [1]) + 2
    table = np.full((len(q_lens), width), 2 ** 31 - 1 if poison else 0, dtype=np.int64)
    kp = np.full((n_pages, page, hkv, d), np.nan if poison else 0.0)
    vp = kp.copy()
    at = 0
    for b, (kv, h) in enumerate(zip(kv_lens, held)):
        table[b, :h] = order[at:at + h]
        at += h
        pos = np.arange(kv)
        pg = table[b, pos // page] if kv else pos
        kp[pg, pos % page] = rng.standard_normal((kv, hkv, d))
        vp[pg, pos % page] = rng.standard_normal((kv, hkv, d))
    n = sum(q_lens)
    q = np.full((n + pad, hq, d), np.nan)
    q[:n] = rng.standard_normal((n, hq, d))
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    to = lambda x, t: torch.from_numpy(np.ascontiguousarray(x)).to(t).to(device)
    return dict(q=to(q, dtype), cu_q=to(cu, torch.int32), kv_len=to(np.array(kv_lens, dtype=np.int64), torch.int32),
                table=to(table, torch.int32), k_pages=to(kp, dtype), v_pages=to(vp, dtype), max_q=max(max(q_lens), 1),
                n=n, q_lens=q_lens, kv_lens=kv_lens, host_table=table)


def check_paged(c, o, lse, what):
    dtype = c["q"].dtype
    qh, kh, vh = (c[x].double().cpu().numpy() for x in ("q", "k_pages", "v_pages"))
    at = 0
    for b, (m, kv) in enumerate(zip(c["q_lens"], c["kv_lens"])):
        if m:
            k, v = (so.paged_keys(x, c["host_table"][b], kv) for x in (kh, vh))
            want = so.attend_rows(qh[at:at + m], k, v, kv - m)
            check_rows(dtype, o[at:at + m], None if lse is None else lse[at:at + m], want, max(kv, 1),
                       f"{what}, request {b} ({m} of {kv})")
        at += m
