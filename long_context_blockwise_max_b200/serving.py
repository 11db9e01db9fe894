"""Python binding of the serving operators (C ABI in ``include/pulsar_serving.h``).

One step of a server over a paged KV cache, for requests of any lengths:

* ``pa_paged_schedule``  page tables, slot map and positions of the step's new
  tokens, built on the GPU from the requests' lengths (once for all layers);
* ``pa_paged_append``    RoPE of the new tokens' Q and K, K and V to the cache;
* ``pa_prompt_attend``   causal attention over packed prompts;
* ``pa_paged_attend``    attention of new tokens (chunks, or one generated token
  each) over the pages.

Argument marshalling only, by the rules of ``pulsar``: shapes, dtypes and
devices are checked here, missing outputs and workspaces allocated with torch,
and raw pointers passed to the C entry point of the same name, on the tensors'
device and its current stream.  No call waits for the GPU (unless
``pulsar.set_status_checks`` is on), so each may be captured into a CUDA graph.
An ordinary call (missing outputs, tensors on the current device) goes through
the compiled call layer ``_serving_call``, which does the same in less time.
"""
from __future__ import annotations

import ctypes
import importlib.util
import os
from functools import lru_cache

import torch

from . import build, pulsar
from .pulsar import PulsarError, _check, _dtype_code, _lib, _need, _same



def _load_call_layer():
    path = build.call_layer_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built; run `python -m long_context_blockwise_max_b200.build`")
    spec = importlib.util.spec_from_file_location(f"{__package__}._serving_call", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


_ordinary = _load_call_layer()

# Every symbol declared in include/pulsar_serving.h.
ABI_SYMBOLS = (
    "pa_paged_schedule_workspace_size", "pa_paged_schedule", "pa_paged_append_workspace_size", "pa_paged_append",
    "pa_prompt_attend_workspace_size", "pa_prompt_attend", "pa_paged_attend_workspace_size", "pa_paged_attend",
)


def _declare():
    P, I32, I64, SZ, D = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_double
    INT = ctypes.c_int
    sig = {
        "pa_paged_schedule_workspace_size": (SZ, [I32]),
        "pa_paged_schedule": (INT, [P, P, I32, P, I64, I32, P, I32, I32, I64, P, P, P, P, P, P, SZ, P]),
        "pa_paged_append_workspace_size": (SZ, [I64]),
        "pa_paged_append": (INT, [P, P, P, INT, I64, I64, I64, I64, I32, I32, I32, D, P, P, P, P, I64, P, P, P, SZ,
                                  P]),
        "pa_prompt_attend_workspace_size": (SZ, [I32, I64, I32, I32, I32, INT]),
        "pa_prompt_attend": (INT, [P, P, P, INT, I64, I64, I64, I64, P, I32, I32, I32, I32, P, P, P, SZ, P]),
        "pa_paged_attend_workspace_size": (SZ, [I32, I64, I32, I32, I32, I32, I32, I32, INT]),
        "pa_paged_attend": (INT, [P, INT, I64, I64, P, P, I32, I32, P, I64, I32, I32, P, P, I32, I32, I32, I32, P, P,
                                  P, SZ, P]),
    }
    # test hook (include/pulsar_testing.h)
    sig["pa_testing_paged_stall"] = (INT, [P, I64, P, P, I32, I32, P, I32, I32, P, P, I32, I32, I32, I32, P, P, SZ, I32,
                                           P])
    for name, (res, args) in sig.items():
        fn = getattr(_lib, name)
        fn.restype, fn.argtypes = res, args


_declare()


def _p(t):
    return None if t is None else t.data_ptr()


def _on(ref: torch.Tensor, *ts):
    """Every tensor (None: skipped) is on ``ref``'s CUDA device."""
    if not ref.is_cuda:
        raise ValueError("tensors must be on a CUDA device")
    dev = ref.device
    for t in ts:
        if t is not None and t.device != dev:
            raise ValueError(f"tensors must be on one CUDA device: {t.device} and {dev}")


def _dense(*named):
    for name, t in named:
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")


def _span(t):
    """First and last byte address of a tensor's elements, or None."""
    if t is None or t.numel() == 0:
        return None
    last = sum((n - 1) * st for n, st in zip(t.shape, t.stride()))
    return t.data_ptr(), t.data_ptr() + (last + 1) * t.element_size() - 1


def _apart(outs, ins):
    """Outputs share no memory with inputs or with one another."""
    for i, (name, out) in enumerate(outs):
        o = _span(out)
        for other, t in list(ins) + list(outs[i + 1:]):
            x = _span(t)
            if o and x and o[0] <= x[1] and x[0] <= o[1]:
                raise ValueError(f"{name}: overlaps {other}")


def _rows(t: torch.Tensor, name: str, d: int | None = None):
    """Packed [N][heads][d] rows, dense inside a token: the token stride."""
    if t.dim() != 3:
        raise ValueError(f"{name}: must be [N][heads][d]")
    n, h, dim = t.shape
    if d is not None and dim != d:
        raise ValueError(f"{name}: head dimension {dim}, expected {d}")
    if t.numel() == 0 or n == 1:
        ld = h * dim
    else:
        ld = t.stride(0)
    if t.numel() and ((dim > 1 and t.stride(2) != 1) or (h > 1 and t.stride(1) != dim)):
        raise ValueError(f"{name}: heads of a token must be dense (strides {tuple(t.stride())})")
    if n > 1 and ld < h * dim:
        raise ValueError(f"{name}: tokens overlap (stride {ld} for {h * dim} elements)")
    return ld


def _ints(named, n):
    for name, t in named:
        _need(t, name, torch.int32, n)
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name}: must be contiguous")


def _table(t: torch.Tensor, B: int):
    """[B][max_pages] int32, dense in a row: the row stride."""
    if t.dim() != 2 or t.dtype != torch.int32:
        raise ValueError("block_table: must be [B][max_pages] int32")
    if t.shape[0] < B:
        raise ValueError(f"block_table: {t.shape[0]} rows for {B} requests")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("block_table: rows must be dense")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError("block_table: rows overlap")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _ws(nbytes: int, ref: torch.Tensor, ws):
    if ws is None:
        return torch.empty(nbytes if nbytes > 256 else 256, dtype=torch.uint8, device=ref.device)
    if not ws.is_contiguous():
        raise ValueError("ws: must be contiguous")
    return ws


def _call(fn, ref: torch.Tensor, ws, *args):
    """The C entry point on ``ref``'s device and that device's current stream."""
    dev = ref.device.index
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _call(fn, ref, ws, *args)
    rc = fn(*args, ws.data_ptr(), ws.numel() * ws.element_size(), torch._C._cuda_getCurrentRawStream(dev))
    if rc != 0 or pulsar._STATUS_CHECKS:
        _check(rc, fn.__name__, ws)


def _answer(got, name: str):
    """The outputs of an ordinary call, or its error."""
    if type(got) is int:
        raise PulsarError(got, name)
    if pulsar._STATUS_CHECKS:
        _check(0, name, got[-1])
    return got


def pa_paged_schedule(q_len, kv_len, block_table, free_pages, page_size: int, n_tokens: int, cu_q=None,
                      kv_len_out=None, positions=None, slots=None, n_used=None, ws=None):
    """Page tables, slot map and positions of one step.  ``q_len``, ``kv_len``
    [B]: new and cached tokens of each request; ``block_table`` [B][max_pages]
    is extended in place from the front of ``free_pages``.  ``n_tokens``: rows
    of the step's tensors (at least sum(q_len); rows behind it get slot -1).
    Returns (cu_q, kv_len_out, positions, slots, n_used, ws)."""
    if cu_q is None and kv_len_out is None and positions is None and slots is None and n_used is None and ws is None:
        got = _ordinary.paged_schedule(q_len, kv_len, block_table, free_pages, page_size, n_tokens)
        if got is not None:
            return _answer(got, "pa_paged_schedule")
    _on(q_len, kv_len, block_table, free_pages, cu_q, kv_len_out, positions, slots, n_used, ws)
    B, n_tokens = q_len.numel(), int(n_tokens)
    _ints((("q_len", q_len), ("kv_len", kv_len), ("kv_len_out", kv_len_out)), B)
    stride = _table(block_table, B)
    _ints((("free_pages", free_pages),), 0)
    _ints((("cu_q", cu_q),), B + 1)
    _ints((("positions", positions), ("slots", slots)), n_tokens)
    _ints((("n_used", n_used),), 1)
    _apart([("kv_len_out", kv_len_out), ("cu_q", cu_q), ("positions", positions), ("slots", slots),
            ("n_used", n_used), ("block_table", block_table)],
           [("q_len", q_len), ("kv_len", kv_len), ("free_pages", free_pages)])
    given = (cu_q, kv_len_out, positions, slots, n_used)
    sizes = (B + 1, B, n_tokens, n_tokens, 1)
    if any(t is None for t in given):   # one allocation for those that are missing
        own = torch.empty(sum(n for n, t in zip(sizes, given) if t is None), dtype=torch.int32, device=q_len.device)
        own = iter(own.split([n for n, t in zip(sizes, given) if t is None]))
        cu_q, kv_len_out, positions, slots, n_used = (next(own) if t is None else t for t in given)
    ws = _ws(256, q_len, ws)
    _call(_lib.pa_paged_schedule, q_len, ws, _p(q_len), _p(kv_len), B, _p(block_table), stride, block_table.shape[1],
          _p(free_pages), free_pages.numel(), int(page_size), n_tokens, _p(cu_q), _p(kv_len_out), _p(positions),
          _p(slots), _p(n_used))
    return cu_q, kv_len_out, positions, slots, n_used, ws


def _pages(k_pages, v_pages, dtype, hkv=None, d=None):
    if k_pages.dim() != 4:
        raise ValueError("k_pages: must be [n_pages][page_size][hkv][d]")
    _same(k_pages, ("v_pages", v_pages))
    _dense(("k_pages", k_pages), ("v_pages", v_pages))
    if k_pages.dtype != dtype:
        raise ValueError(f"k_pages: dtype {k_pages.dtype}, expected {dtype}")
    if hkv is not None and k_pages.shape[2] != hkv:
        raise ValueError(f"k_pages: {k_pages.shape[2]} kv heads, expected {hkv}")
    if d is not None and k_pages.shape[3] != d:
        raise ValueError(f"k_pages: head dimension {k_pages.shape[3]}, expected {d}")


def pa_paged_append(q, k_new, v_new, positions, slots, k_pages, v_pages, rope_theta: float = 0.0, q_out=None,
                    k_out=None, want_k: bool = False, ws=None):
    """Rotate the new tokens' ``q`` [N][hq][d] (or None) and ``k_new``
    [N][hkv][d] at ``positions`` (``rope_theta`` 0: not rotated) and write K
    and ``v_new`` to ``slots`` of the cache (``slots``, ``k_pages`` and
    ``v_pages`` None: nothing is written; negative slots are skipped).  Returns
    (rotated q or None, rotated k or None, ws); ``want_k`` or ``k_out`` asks
    for k."""
    if q_out is None and k_out is None and ws is None:
        got = _ordinary.paged_append(q, k_new, v_new, positions, slots, k_pages, v_pages, rope_theta, want_k)
        if got is not None:
            return _answer(got, "pa_paged_append")
    _on(k_new, q, v_new, positions, slots, k_pages, v_pages, q_out, k_out, ws)
    ldk = _rows(k_new, "k_new")
    N, hkv, d = k_new.shape
    ldq = ldv = 0
    hq = hkv
    if q is not None:
        ldq = _rows(q, "q", d)
        hq = q.shape[1]
        if q.shape[0] != N or q.dtype != k_new.dtype:
            raise ValueError(f"q: {q.dtype} {tuple(q.shape)} does not match k_new {k_new.dtype} {tuple(k_new.shape)}")
    elif q_out is not None:
        raise ValueError("q_out: given without q")
    if (slots is None) != (k_pages is None) or (slots is None) != (v_pages is None):
        raise ValueError("slots, k_pages and v_pages must be given together")
    n_slots = 0
    if slots is not None:
        _same(k_new, ("v_new", v_new))
        if v_new is None:
            raise ValueError("v_new: needed to append")
        ldv = _rows(v_new, "v_new", d)
        _pages(k_pages, v_pages, k_new.dtype, hkv, d)
        n_slots = k_pages.shape[0] * k_pages.shape[1]
    _ints((("positions", positions), ("slots", slots)), N)
    if rope_theta and positions is None:
        raise ValueError("positions: needed to rotate")
    _need(q_out, "q_out", k_new.dtype, N * hq * d)
    _need(k_out, "k_out", k_new.dtype, N * hkv * d)
    if q_out is not None or k_out is not None:
        _dense(("q_out", q_out), ("k_out", k_out))
    ins = [("q", q), ("k_new", k_new), ("v_new", v_new), ("positions", positions), ("slots", slots)]
    pages = [("k_pages", k_pages), ("v_pages", v_pages)]
    for name, out, src, ld in (("q_out", q_out, q, ldq), ("k_out", k_out, k_new, ldk)):
        here = out is not None and src is not None and out.data_ptr() == src.data_ptr()
        if here and N > 1 and ld != src.shape[1] * d:
            raise ValueError(f"{name}: in place only for dense rows")
        _apart([(name, out)], [i for i in ins if not (here and i[1] is src)] + pages)
    _apart([("q_out", q_out), ("k_out", k_out)], ())
    if N > 0:
        _apart(pages, ins)
    if q is not None and q_out is None:
        q_out = torch.empty((N, hq, d), dtype=q.dtype, device=q.device)
    if k_out is None and want_k:
        k_out = torch.empty((N, hkv, d), dtype=k_new.dtype, device=k_new.device)
    ws = _ws(256, k_new, ws)
    _call(_lib.pa_paged_append, k_new, ws, _p(q), _p(k_new), _p(v_new), _dtype_code(k_new), N, ldq, ldk, ldv, hq, hkv,
          d, float(rope_theta), _p(positions), _p(slots), _p(k_pages), _p(v_pages), n_slots, _p(q_out), _p(k_out))
    return q_out, k_out, ws


def _attend_outputs(q, o, lse, want_lse, ins):
    N, hq, d = q.shape
    if o is not None and N > 0 and o.data_ptr() == q.data_ptr():
        raise ValueError("o: must not be q")
    if o is not None or lse is not None:
        _apart([("o", o), ("lse", lse)], ins)
    _need(o, "o", q.dtype, N * hq * d)
    _need(lse, "lse", torch.float32, N * hq)
    _dense(("o", o), ("lse", lse))
    if o is None:
        o = torch.empty((N, hq, d), dtype=q.dtype, device=q.device)
    if lse is None and want_lse:
        lse = torch.empty((N, hq), dtype=torch.float32, device=q.device)
    return o, lse


def _batch(cu_q):
    _ints((("cu_q", cu_q),), 1)
    return cu_q.numel() - 1


@lru_cache(maxsize=4096)   # a pure function of sizes
def pa_prompt_attend_workspace_size(B, N, hq, hkv, d, dtype) -> int:
    return _lib.pa_prompt_attend_workspace_size(B, N, hq, hkv, d, dtype)


def pa_prompt_attend(q, k, v, cu_q, o=None, lse=None, want_lse: bool = True, ws=None):
    """Causal attention over packed prompts: rows ``cu_q[b]`` ..
    ``cu_q[b + 1] - 1`` of ``q`` [N][hq][d], ``k`` and ``v`` [N][hkv][d]
    (rotated) are prompt b.  Rows behind the last prompt are left as they
    were.  Returns (o, lse or None, ws)."""
    if o is None and lse is None and ws is None:
        got = _ordinary.prompt_attend(q, k, v, cu_q, want_lse)
        if got is not None:
            return _answer(got, "pa_prompt_attend")
    _on(q, k, v, cu_q, o, lse, ws)
    ldq = _rows(q, "q")
    N, hq, d = q.shape
    ldk, ldv = _rows(k, "k", d), _rows(v, "v", d)
    _same(k, ("v", v))
    if k.shape[0] != N or k.dtype != q.dtype:
        raise ValueError(f"k: {k.dtype} {tuple(k.shape)} does not match q {q.dtype} {tuple(q.shape)}")
    hkv, B, dt = k.shape[1], _batch(cu_q), _dtype_code(q)
    o, lse = _attend_outputs(q, o, lse, want_lse, [("q", q), ("k", k), ("v", v), ("cu_q", cu_q)])
    if ws is None:
        ws = _ws(pa_prompt_attend_workspace_size(B, N, hq, hkv, d, dt), q, None)
    ws = _ws(0, q, ws)
    _call(_lib.pa_prompt_attend, q, ws, _p(q), _p(k), _p(v), dt, N, ldq, ldk, ldv, _p(cu_q), B, hq, hkv, d, _p(o),
          _p(lse))
    return o, lse, ws


@lru_cache(maxsize=4096)
def pa_paged_attend_workspace_size(B, N, max_q, max_pages, page_size, hq, hkv, d, dtype) -> int:
    return _lib.pa_paged_attend_workspace_size(B, N, max_q, max_pages, page_size, hq, hkv, d, dtype)


def pa_paged_attend(q, cu_q, kv_len, block_table, k_pages, v_pages, max_q: int, o=None, lse=None,
                    want_lse: bool = True, ws=None):
    """Attention of packed new tokens ``q`` [N][hq][d] (rotated) over each
    request's pages: token i of request b, at position kv_len[b] - q_len[b] +
    i, sees the keys up to its own.  ``kv_len`` [B] counts the new tokens (they
    are in the cache already); ``max_q`` bounds the new tokens of a request.
    Rows behind the last request are left as they were.  Returns (o, lse or
    None, ws)."""
    if o is None and lse is None and ws is None:
        got = _ordinary.paged_attend(q, cu_q, kv_len, block_table, k_pages, v_pages, max_q, want_lse)
        if got is not None:
            return _answer(got, "pa_paged_attend")
    _on(q, cu_q, kv_len, block_table, k_pages, v_pages, o, lse, ws)
    ldq = _rows(q, "q")
    N, hq, d = q.shape
    B, dt = _batch(cu_q), _dtype_code(q)
    _ints((("kv_len", kv_len),), B)
    stride = _table(block_table, B)
    _pages(k_pages, v_pages, q.dtype, None, d)
    n_pages, page_size, hkv, _ = k_pages.shape
    o, lse = _attend_outputs(q, o, lse, want_lse,
                             [("q", q), ("cu_q", cu_q), ("kv_len", kv_len), ("block_table", block_table),
                              ("k_pages", k_pages), ("v_pages", v_pages)])
    if ws is None:
        ws = _ws(pa_paged_attend_workspace_size(B, N, int(max_q), block_table.shape[1], page_size, hq, hkv, d, dt),
                 q, None)
    ws = _ws(0, q, ws)
    _call(_lib.pa_paged_attend, q, ws, _p(q), dt, N, ldq, _p(cu_q), _p(kv_len), B, int(max_q), _p(block_table), stride,
          block_table.shape[1], page_size, _p(k_pages), _p(v_pages), n_pages, hq, hkv, d, _p(o), _p(lse))
    return o, lse, ws


def pa_testing_paged_stall(q, cu_q, kv_len, block_table, k_pages, v_pages, max_q: int, wait_limit_us: int):
    """Test hook: ``pa_paged_attend`` (bf16, dense tensors) with one
    unsatisfiable barrier per block and waits limited to ``wait_limit_us``; the
    workspace status then reads PA_ERR_TIMEOUT.  Returns the workspace."""
    _on(q, cu_q, kv_len, block_table, k_pages, v_pages)
    N, hq, d = q.shape
    n_pages, page_size, hkv, _ = k_pages.shape
    B, width = _batch(cu_q), block_table.shape[1]
    o = torch.empty_like(q)
    ws = _ws(pa_paged_attend_workspace_size(B, N, int(max_q), width, page_size, hq, hkv, d, pulsar.PA_BF16), q, None)
    rc = _lib.pa_testing_paged_stall(_p(q), N, _p(cu_q), _p(kv_len), B, int(max_q), _p(block_table), width, page_size,
                                     _p(k_pages), _p(v_pages), n_pages, hq, hkv, d, _p(o), _p(ws), ws.numel(),
                                     int(wait_limit_us), torch.cuda.current_stream(q.device).cuda_stream)
    _check(rc, "pa_testing_paged_stall")
    return ws
