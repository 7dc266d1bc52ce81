"""The largest and smallest sizes of the attention calls, as far as the host decides (no GPU)."""
import pytest

from ivf_top_key_b200 import _capi as C

P = 1 << 20   # an aligned address that nothing follows


@pytest.mark.parametrize("total_q,total_k", [(4, 2 ** 31 - 1), (4, 2 ** 31 - 256), (2 ** 31 - 256, 4)])
def test_more_tokens_than_tiles_can_count_are_refused(total_q, total_k):
    with pytest.raises(C.AiError, match="2\\^31 - 257 tokens") as e:
        C.ai_attend_prompt(P, (512, 128), P, (256, 128), P, (256, 128), P, P, 1, total_q, total_k, 4, 2, 128, 1.0, P, None,
                           None, None, 0, 0)
    assert e.value.code == -1


def test_no_rows_are_attended_without_ids():
    """An empty list of ids is a null pointer, and nothing is launched for it."""
    c = C.AiCache(k=P, v=P, tables=P, lens=P, dtype=C.AI_BF16, n_layers=1, n_pages=8, page_size=16, n_kv_heads=2,
                  head_dim=128, n_seqs=3, max_pages=4)
    before = C.ai_kernel_launches()
    C.ai_attend_selected(c, 0, None, None, 0, 7, 4, None, 1.0, None, None, P, 1 << 40, 0)
    C.ai_attend_cached(c, 0, None, 0, 4, None, 1.0, None, None, P, 1 << 40, 0)
    assert C.ai_kernel_launches() == before
    with pytest.raises(C.AiError, match="null"):
        C.ai_attend_selected(c, 0, P, None, 3, 7, 4, None, 1.0, P, None, P, 1 << 40, 0)
