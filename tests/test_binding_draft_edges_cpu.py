"""The binding's calls for drafted tokens without a GPU: tensors without elements."""
import pytest
import torch

import token_level_sparse_gb300 as T
from test_binding_cpu import Reached, _on, context  # noqa: F401
from test_binding_draft_cpu import B, BF, D, H, HKV, I32, ROWS, _calls, page_bytes  # noqa: F401


def test_a_mask_without_words_is_no_missing_mask(context):  # noqa: F811
    """Its address is NULL, which stands for drafts that see those up to their own: refused, where there are rows."""
    c = context(H, HKV, D, T.TS_KV_BF16, B, 4, 8)
    call, good = _calls(c)["tree_attend"]
    good = {key: _on(t) for key, t in good.items()}
    with pytest.raises(T.TokenSelectError) as e:
        call(**(good | dict(mask=_on(torch.zeros(ROWS, 0, dtype=I32)))))
    assert e.value.status == T.STATUS_CODE["TS_ERR_SHAPE"]
    none = _on(torch.zeros(0, H, D, dtype=BF))
    for words in (0, 1):                                           # a batch without drafts has nothing to mask
        with pytest.raises(Reached):
            call(**(good | dict(q=none, out=none, lse=_on(torch.zeros(0, H)), mask=_on(torch.zeros(0, words, dtype=I32)))))
