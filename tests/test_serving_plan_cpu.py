"""Which kernels an attention call over pages has, as its workspace shows it."""
import pytest

from long_context_blockwise_max_b200 import build


@pytest.fixture(scope="module")
def size():
    build.build()
    from long_context_blockwise_max_b200 import serving
    # (caches long enough for the most partial results of the tile kernel, whatever N)
    return lambda N, hq, hkv, max_q=64, B=4: serving.pa_paged_attend_workspace_size(B, N, max_q, 8192, 16, hq, hkv, 128, 1)


@pytest.mark.parametrize("hq,hkv", [(32, 8), (16, 2), (16, 1), (32, 1), (64, 1), (34, 2)])
def test_decode_scratch_only_where_a_request_can_be_short_enough(size, hq, hkv):
    # 148 blocks' partial results of 16 rows, 2.4 MB: in a ragged call, unless one
    # token has more rows than that
    ragged, uniform = size(4 * 64 - 1, hq, hkv), size(4 * 64, hq, hkv)
    scratch = 148 * 2 * 16 * 129 * 4
    if hq // hkv <= 16:
        assert scratch <= ragged - uniform < 2 * scratch
    else:
        assert abs(ragged - uniform) < scratch // 8
