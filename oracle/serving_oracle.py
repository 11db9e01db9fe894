"""fp64 / integer oracle of the serving operators (numpy, host only).

The definitions of ``include/pulsar_serving.h`` written out request by
request: page tables and slot maps by a loop over requests and tokens, RoPE
by complex rotation, attention by an explicit mask and a softmax in fp64.
"""
import numpy as np


def schedule_step(q_len, kv_len, table, free_pages, page_size, n_tokens):
    """Returns (cu_q, kv_len_out, positions, slots, n_used, table, refused).
    ``table`` is copied.  Lengths are non-negative."""
    table = np.array(table, dtype=np.int64, copy=True)
    max_pages = table.shape[1]
    cu = np.zeros(len(q_len) + 1, dtype=np.int64)
    kv_out = np.array(kv_len, dtype=np.int64)
    pos = np.zeros(n_tokens, dtype=np.int64)
    slots = np.full(n_tokens, -1, dtype=np.int64)
    asked, used, refused = 0, 0, []
    for b, (q, kv) in enumerate(zip(q_len, kv_len)):
        cu[b + 1] = cu[b] + q
        held = -(-kv // page_size)
        need = -(-(kv + q) // page_size) - held if q > 0 else 0
        ok = q == 0 or held + need <= max_pages
        first = asked
        if ok:
            asked += need
            ok = need == 0 or asked <= len(free_pages)
        if ok and need:
            table[b, held:held + need] = free_pages[first:first + need]
            used = asked
        if ok:
            kv_out[b] = kv + q
        elif q > 0:
            refused.append(b)
        for i in range(q):
            t = cu[b] + i
            if t >= n_tokens:
                break
            p = kv + i
            pos[t] = p
            if ok:
                slots[t] = table[b, p // page_size] * page_size + p % page_size
    return cu, kv_out, pos, slots, used, table, refused


def rope(x, positions, theta):
    """Rotate-half RoPE of [N][h][d] rows in fp64 (theta 0: unchanged)."""
    x = np.asarray(x, dtype=np.float64)
    if theta == 0:
        return x
    half = x.shape[-1] // 2
    omega = theta ** (-2.0 * np.arange(half) / x.shape[-1])
    turn = np.exp(1j * np.asarray(positions, dtype=np.float64)[:, None, None] * omega)
    z = (x[..., :half] + 1j * x[..., half:]) * turn
    return np.concatenate([z.real, z.imag], -1)


def attend_rows(q, k, v, first):
    """q [n][hq][d], k and v [T][hkv][d]; row i sees keys 0 .. first + i.
    Returns (o, lse, mag, raw): mag = sum_j p_ij |v_j| (what a relative error of
    the probabilities is multiplied by) and raw = max sum |q_m k_m| / sqrt(d)
    over the visible keys (what a rounding of the products is relative to)."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    n, hq, d = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    o, mag = np.zeros_like(q), np.zeros_like(q)
    lse = np.full((n, hq), -np.inf)
    raw = 0.0
    for i in range(n):
        m = min(first + i + 1, k.shape[0])
        if m <= 0:
            continue
        for h in range(hkv):
            qi = q[i, h * g:(h + 1) * g]
            s = qi @ k[:m, h].T / np.sqrt(d)
            raw = max(raw, float((np.abs(qi) @ np.abs(k[:m, h]).T).max() / np.sqrt(d)))
            top = s.max(-1, keepdims=True)
            e = np.exp(s - top)
            z = e.sum(-1, keepdims=True)
            p = e / z
            o[i, h * g:(h + 1) * g] = p @ v[:m, h]
            mag[i, h * g:(h + 1) * g] = p @ np.abs(v[:m, h])
            lse[i, h * g:(h + 1) * g] = (top + np.log(z))[:, 0]
    return o, lse, mag, raw


def paged_keys(pages, table_row, length):
    """The first ``length`` rows of a request's cache, [length][hkv][d]."""
    p = pages.shape[1]
    at = np.arange(length)
    return pages[np.asarray(table_row)[at // p], at % p]
