"""The attention and cache calls at their edges: what lists ask for, values that are not finite, shared pages, long rows,
tensors that are dropped after the call."""
import pytest
import torch

from tests import attention_ref as R

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a GPU", allow_module_level=True)

from ivf_top_key_b200 import AiError, PagedCache  # noqa: E402
from tests.test_gpu_attention import _i32  # noqa: E402


@pytest.mark.parametrize("asked", [0, 80, 96, 97, 112, 128, 129, 144, 256])
def test_extend_that_needs_no_page_is_done_whatever_the_list_asks(asked):
    """Eight pages, six of them free: sequences 1 and 3 have room in their own part page."""
    c = PagedCache(n_pages=8, page_size=16, n_kv_heads=1, head_dim=64, n_seqs=4, max_pages=16)
    ref = R.Pages(8, 16, 4, 16)
    for seqs, counts in (([1, 3], [5, 1]), ([0, 1, 2, 3], [asked, 1, 1, 15])):
        ref.extend(seqs, counts)
        c.extend(_i32(seqs), _i32(counts))
        ref.same_as(c)
    assert ref.lens[1] == 6 and ref.lens[3] == 16
    if asked > 80:   # six free pages, one of them for sequence 2
        with pytest.raises(AiError, match="OOM"):
            c.check()
    c.check()


def test_extend_decode_steps_beside_one_request_beyond_the_cache():
    """The same in a list of more than one pass of the planning block."""
    n = 1500
    c = PagedCache(n_pages=2 * n, page_size=2, n_kv_heads=1, head_dim=64, n_seqs=n, max_pages=2 * n + 1)
    ref = R.Pages(2 * n, 2, n, 2 * n + 1)
    for seqs, counts in ((range(1, n), [1 + s % 2 for s in range(1, n)]), (range(n), [4 * n + 1] + [1] * (n - 1))):
        ref.extend(list(seqs), counts)
        c.extend(_i32(list(seqs)), _i32(counts))
        ref.same_as(c)
    assert ref.lens[:5] == [0, 2, 2, 2, 2]
