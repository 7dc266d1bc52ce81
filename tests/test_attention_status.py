"""What the status word of the attention and cache calls tells a caller (no GPU: the bits are set here)."""
import os
import re

import pytest
import torch

from ivf_top_key_b200 import AiError, PagedCache
from ivf_top_key_b200 import _capi as C


def _cache_with(bits):
    c = object.__new__(PagedCache)   # without its tensors on a GPU
    c.status = torch.tensor([bits], dtype=torch.int32)
    return c


@pytest.mark.parametrize("bits,code", [
    (C.AI_DEVFLAG_TIMEOUT, -5), (C.AI_DEVFLAG_RANGE, -4), (C.AI_DEVFLAG_CAPACITY, -2),
    (C.AI_DEVFLAG_TIMEOUT | C.AI_DEVFLAG_RANGE, -5), (C.AI_DEVFLAG_TIMEOUT | C.AI_DEVFLAG_CAPACITY, -5),
    (C.AI_DEVFLAG_RANGE | C.AI_DEVFLAG_CAPACITY, -4),
])
def test_check_raises_for_what_happened(bits, code):
    c = _cache_with(bits)
    with pytest.raises(AiError) as e:
        c.check()
    assert e.value.code == code
    assert ("not valid" in str(e.value)) == (code == -5)
    c.check()   # once


def test_check_of_a_clean_word():
    _cache_with(0).check()


def test_bits_match_the_header():
    src = open(os.path.join(os.path.dirname(os.path.dirname(__file__)), "include", "ai_index.h")).read()
    for name, bit in re.findall(r"#define (AI_DEVFLAG_\w+) (\d+)", src):
        assert getattr(C, name) == int(bit)
