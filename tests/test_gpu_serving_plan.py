"""What the plan of an attention call decides, read from its workspace: the
status block is followed by the plan's head, whose first words are the number of
pieces of the tile kernel, the number of row groups whose keys were cut, an abort
flag, and whether pieces are taken over all kv heads in order of depth."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def S():
    from long_context_blockwise_max_b200 import serving
    assert torch.cuda.is_available()
    return serving


def plan_of(S, q_lens, kv_lens, hq=32, hkv=8, d=128, page=16):
    """(pieces, row groups cut, over all heads) of a paged call; requests share pages."""
    width = max(-(-kv // page) for kv in kv_lens)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cu = [0]
    for m in q_lens:
        cu.append(cu[-1] + m)
    pages = torch.zeros((2, width, page, hkv, d), dtype=torch.bfloat16, device="cuda")
    table = torch.arange(width, dtype=torch.int32, device="cuda").repeat(len(q_lens), 1)
    q = torch.zeros((cu[-1], hq, d), dtype=torch.bfloat16, device="cuda")
    _, lse, ws = S.pa_paged_attend(q, i32(cu), i32(kv_lens), table, pages[0], pages[1], max(q_lens))
    assert S.pulsar.pa_workspace_status(ws) == 0
    # all scores are zero: lse is the logarithm of the number of keys
    at = torch.cat([torch.arange(kv - m + 1, kv + 1) for m, kv in zip(q_lens, kv_lens)]).double().log()
    assert (lse.double().cpu() - at[:, None]).abs().max() <= 1e-4
    pieces, cut, _, inner = ws[256:272].view(torch.int32).tolist()
    return pieces, cut, inner


@pytest.mark.parametrize("chunks,tokens,tiles", [(1, 2, True), (1, 8, False), (2, 2, True), (2, 8, False), (4, 2, True),
                                                 (4, 4, False), (6, 8, True)])
def test_few_tokens_take_no_blocks_that_the_chunks_need(S, chunks, tokens, tiles):
    q = [256] * chunks + [1] * tokens
    both = plan_of(S, q, [8000] * chunks + [64] * tokens)
    alone = plan_of(S, q[:chunks], [8000] * chunks)
    whole = 4 * chunks
    assert both[0] >= whole and alone[0] >= whole
    # the tokens are pieces of their own, or the chunks' pieces are what they are without them
    if tiles:
        assert both[0] - both[1] >= tokens and both[0] > whole
    else:
        assert both == alone


@pytest.mark.parametrize("others,keys,cut", [(40, 8192, False), (40, 32768, True), (64, 8192, False), (64, 32768, True),
                                             (140, 32768, False), (140, 131072, True)])
def test_among_many_rows_a_cut_has_to_promise_enough(S, others, keys, cut):
    pieces, groups, _ = plan_of(S, [512] + [128] * others, [keys] + [1024] * others)
    assert pieces >= 8 + 2 * others
    assert (groups > 0) == cut


@pytest.mark.parametrize("q,kv,inner", [([2048] * 8, [32768] * 8, 0), ([2048] * 4, [65536, 32768, 21845, 16384], 1),
                                        ([16384], [32768], 0), ([64, 64, 200, 1000], [20000, 4000, 300, 8000], 1)])
def test_even_pieces_of_a_head_share_its_keys(S, q, kv, inner):
    # beyond what L2 holds (or below it: the last case), in no more than two waves a head
    assert plan_of(S, q, kv)[2] == inner
