"""The 4-bit cache's calls at the edges of what they take, on a GPU: selections, non-finite and huge queries, values next
to fp16's largest, groups of very different size, waits that run out, ties, graphs that run at once."""
import math

import numpy as np
import pytest
import torch

import oracle as O
from mixed_bit_kv_gb300 import rdkv
from test_gpu_q4 import DEV, TYPES, _cache, _check_attention, _filled, _rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if DEV is None:
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()


# ---------------------------------------------------------------- selections
@pytest.mark.parametrize("T", [1, 3])
def test_an_empty_or_misshapen_selection_is_refused(T):
    """Not taken for every position, and not for another order of the same numbers."""
    c, kh, vh = _filled([200, 70], 2, 64, torch.float16)
    q = _rows(2 * T, 4, 64, torch.float16, 9).view(2, T, 4, 64)
    out = torch.full(q.shape, 7.0, dtype=torch.float16, device=DEV)
    sel = torch.zeros(2, T, 2, 4, dtype=torch.int32, device=DEV)
    for bad in (sel[..., :0], torch.empty(2, T, 2, 0, dtype=torch.int32, device=DEV), sel.view(2, 2, T, 4) if T > 1 else sel.view(1, 2, 2, 4),
                sel.view(-1, 4)):
        with pytest.raises(rdkv.RDKVError):
            rdkv.rdkv_q4_attn(c, q.to(DEV), sel=bad, out=out)
    assert (out == 7).all()
    sel[:] = -1                                    # a selection of no page that has a size: nothing is seen
    o, lse = rdkv.rdkv_q4_attn(c, q.to(DEV), sel=sel)
    assert (o == 0).all() and (lse == -math.inf).all() and rdkv.rdkv_q4_status(c) == 0
