"""Sizes that the prompt call refuses before anything is launched (no GPU)."""
import pytest

from ivf_top_key_b200 import _capi as C

P = 1 << 20   # an aligned address that nothing follows


@pytest.mark.parametrize("total_q,total_k", [(4, 2 ** 31 - 1), (4, 2 ** 31 - 256), (2 ** 31 - 256, 4)])
def test_more_tokens_than_tiles_can_count_are_refused(total_q, total_k):
    with pytest.raises(C.AiError, match="2\\^31 - 257 tokens") as e:
        C.ai_attend_prompt(P, (512, 128), P, (256, 128), P, (256, 128), P, P, 1, total_q, total_k, 4, 2, 128, 1.0, P, None,
                           None, None, 0, 0)
    assert e.value.code == -1
