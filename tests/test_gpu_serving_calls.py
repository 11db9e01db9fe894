"""The serving operators' calls from Python on CUDA tensors: what the ordinary
call refuses, raises and leaves to other threads."""
import threading
import time

import pytest
import torch

from serving_cases import randn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from long_context_blockwise_max_b200 import serving
    assert torch.cuda.is_available()
    return serving


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def test_the_ordinary_append_refuses_pages_over_its_inputs(S):
    bf = torch.bfloat16
    both = torch.zeros(2 * 6 * 16 * 2 * 64 + 64, dtype=bf, device="cuda")
    size = 6 * 16 * 2 * 64
    kp, vp = both[:size].view(6, 16, 2, 64), both[size:2 * size].view(6, 16, 2, 64)
    q, k, v = randn((10, 8, 64), bf, 1), randn((10, 2, 64), bf, 2), randn((10, 2, 64), bf, 3)
    pos, slots = i32(range(10)), i32(range(20, 30))

    def bad(match, *args):
        with pytest.raises(ValueError, match=match):
            S.pa_paged_append(*args, rope_theta=1e4)
    bad("k_pages: overlaps v_pages", q, k, v, pos, slots, kp, kp)
    bad("k_pages: overlaps v_pages", q, k, v, pos, slots, kp, both[size - 64:2 * size - 64].view(6, 16, 2, 64))
    for pages, name in ((kp, "k_pages"), (vp, "v_pages")):
        rows = pages.view(-1, 2, 64)
        bad(f"{name}: overlaps k_new", q, rows[86:96], v, pos, slots, kp, vp)
        bad(f"{name}: overlaps v_new", q, k, rows[:10], pos, slots, kp, vp)
        bad(f"{name}: overlaps q", pages.view(-1, 8, 64)[14:24], k, v, pos, slots, kp, vp)
        bad(f"{name}: overlaps positions", q, k, v, rows.view(torch.int32).view(-1)[-10:], slots, kp, vp)
        bad(f"{name}: overlaps slots", q, k, v, pos, rows.view(torch.int32).view(-1)[:10], kp, vp)
    # neighbours do not overlap
    assert both.eq(0).all()
    qr, _, ws = S.pa_paged_append(q, k, v, pos, slots, kp, vp, rope_theta=1e4)
    assert S.pulsar.pa_workspace_status(ws) == 0
    assert torch.equal(vp.view(-1, 2, 64)[20:30], v) and both[2 * size:].eq(0).all() and both[:20 * 128].eq(0).all()


def test_the_ordinary_schedule_refuses_a_table_over_its_inputs(S):
    ints = torch.arange(40, dtype=torch.int32, device="cuda")
    before = ints.clone()
    table, other = ints[8:24].view(2, 8), i32([3, 4])

    def bad(match, *args):
        with pytest.raises(ValueError, match=match):
            S.pa_paged_schedule(*args, 16, 4)
    bad("block_table: overlaps q_len", ints[7:9], other, table, ints[30:])
    bad("block_table: overlaps kv_len", other, ints[23:25], table, ints[30:])
    bad("block_table: overlaps free_pages", other, other, table, ints[20:])
    bad("block_table: overlaps free_pages", other, other, ints[8:24].view(2, 8)[:, :4], ints[15:20])
    torch.cuda.synchronize()
    assert torch.equal(ints, before)
    cu, kv, pos, slots, used, ws = S.pa_paged_schedule(other, ints[:2], table, ints[24:], 16, 7)
    assert S.pulsar.pa_workspace_status(ws) == 0 and cu.tolist() == [0, 3, 7] and used.tolist() == [1]


def test_an_allocation_that_fails_raises_what_torch_raises(S):
    lens, table = i32([3]), i32([[0, 0]])
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(0.02)      # below 4 GB; the call asks for 8 GB
    try:
        with pytest.raises(torch.OutOfMemoryError):
            S.pa_paged_schedule(lens, i32([0]), table, i32([0, 1]), 16, 2 ** 30)
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    cu, kv, _, _, _, _ = S.pa_paged_schedule(lens, i32([0]), table, i32([0, 1]), 16, 3)
    assert cu.tolist() == [0, 3] and kv.tolist() == [3]


class Undecided:
    def __bool__(self):
        raise KeyError("neither")


def test_a_choice_without_a_truth_value_raises_its_own_error(S):
    q, k = randn((4, 4, 64), torch.bfloat16, 1), randn((4, 2, 64), torch.bfloat16, 2)
    pages = torch.zeros((2, 1, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    row = i32(range(4))
    for call in (lambda: S.pa_prompt_attend(q, k, k, i32([0, 4]), want_lse=Undecided()),
                 lambda: S.pa_paged_attend(q, i32([0, 4]), i32([4]), i32([[0]]), pages[0], pages[1], 4,
                                           want_lse=Undecided()),
                 lambda: S.pa_paged_append(q, k, k, row, row, pages[0], pages[1], rope_theta=1e4, want_k=Undecided())):
        with pytest.raises(KeyError, match="neither"):
            call()


def test_other_threads_run_while_launches_wait(S):
    # the GPU is busy for a second, the queue of launches fills, and a call waits
    # in the launch: not with the interpreter's lock
    lens, table, free = i32([1, 1]), i32([[0, 0], [1, 1]]), i32([5, 6])
    q, k = randn((2, 4, 64), torch.bfloat16, 1), randn((2, 2, 64), torch.bfloat16, 2)
    pages = torch.zeros((2, 2, 16, 2, 64), dtype=torch.bfloat16, device="cuda")
    cu, slots = i32([0, 1, 2]), i32([0, 16])
    calls = (lambda: S.pa_paged_schedule(lens, lens, table, free, 16, 2),
             lambda: S.pa_paged_append(q, k, k, lens, slots, pages[0], pages[1], rope_theta=1e4),
             lambda: S.pa_prompt_attend(q, k, k, cu),
             lambda: S.pa_paged_attend(q, cu, lens, table, pages[0], pages[1], 1))
    for call in calls:
        for _ in range(3):
            call()
        torch.cuda.synchronize()
        stop, gaps = threading.Event(), [0.0]

        def tick():
            last = time.perf_counter()
            while not stop.is_set():
                time.sleep(0.002)
                now = time.perf_counter()
                gaps.append(now - last)
                last = now
        thread = threading.Thread(target=tick)
        thread.start()
        torch.cuda._sleep(2_000_000_000)
        begin = time.perf_counter()
        for _ in range(2500):
            call()
        waited = time.perf_counter() - begin
        stop.set()
        thread.join()
        torch.cuda.synchronize()
        assert waited > 0.4, "no launch had to wait"
        assert max(gaps) < 0.2, f"another thread stood still for {max(gaps):.2f} of {waited:.2f} s"


@pytest.mark.parametrize("captured", [False, True], ids=["eager", "captured"])
def test_a_call_waits_for_what_another_stream_has_to_give(S, captured):
    # q, the lengths and the pages come late from another stream; the calls' kernels,
    # which are set up early, read them only then
    gen = torch.Generator(device="cuda").manual_seed(3)
    rn = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()
    new = dict(x=rn(70, 12, 64), q_len=i32([1, 64, 5]), kv=i32([29, 136, 85]), kp=rn(40, 16, 2, 64), vp=rn(40, 16, 2, 64))
    now = {k: torch.zeros_like(t) if t.dtype == torch.bfloat16 else i32([1, 1, 1]) for k, t in new.items()}
    table, free = torch.arange(39, dtype=torch.int32, device="cuda").view(3, 13), i32(range(39))
    other = torch.cuda.Stream()

    def step(src):
        cu, kv, pos, slots, _, w0 = S.pa_paged_schedule(src["q_len"], src["kv"], table, free, 16, 70)
        q, _, w1 = S.pa_paged_append(src["x"][:, :8], src["x"][:, 8:10], src["x"][:, 10:], pos, slots, src["kp"], src["vp"],
                                     rope_theta=1e4)
        o, lse, w2 = S.pa_paged_attend(q, cu, kv, table, src["kp"], src["vp"], 64)
        p, _, w3 = S.pa_prompt_attend(q, src["x"][:, 8:10], src["x"][:, 10:], cu)
        return o, lse, p, slots, w0, w1, w2, w3

    def late():
        main = torch.cuda.current_stream()
        other.wait_stream(main)
        with torch.cuda.stream(other):
            torch.cuda._sleep(20_000_000)
            for k in new:
                now[k].copy_(new[k])
        main.wait_stream(other)
        return step(now)
    want = step({k: t.clone() for k, t in new.items()})
    again = {k: t.clone() for k, t in now.items()}
    step(again)
    torch.cuda.synchronize()
    if captured:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = late()
    for _ in range(2):
        for k, t in now.items():
            t.copy_(torch.zeros_like(t) if t.dtype == torch.bfloat16 else i32([1, 1, 1]))
        if captured:
            g.replay()
        else:
            got = late()
        torch.cuda.synchronize()
        assert all(S.pulsar.pa_workspace_status(w) == 0 for w in got[4:])
        for a, b in zip(got[:4], want[:4]):
            assert torch.equal(a, b)
