"""Outputs that nothing would write are refused, not left as they were (host side, no GPU)."""
import pytest
import torch

import context_attention_partial_gb300 as cp
from test_abi import FAKE, NULL, t
from test_cache_abi import F32, FAR, append, arr, dims


def test_queries_out_without_queries():
    assert append(q=None, q_out=t((2, 4, 3, 64), data=FAR)) == NULL
    e = t((2, 2, 0, 64), data=0)
    assert append(k=e, v=e, q_out=t((2, 4, 0, 64), data=0)) == NULL
    x, pages = torch.zeros(1, 1, 4, 64), torch.zeros(2, 1, 16, 64)
    i, n = torch.zeros(1, 2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(cp.CpattnError) as e:
        cp.cache_append(x, x, pages, pages, i, n, q_out=x)
    assert e.value.name == "CPATTN_ERR_NULL"


def test_weights_gradients_without_weights():
    x, pos = arr([t((1, 4, 16, 128))]), t((16, 1), F32)
    assert cp.load_library().cpattn_norm_rotary_backward(1, x, None, 1e-6, pos, 1, dims((128,)), 1e4, 1, x,
                                                         arr([t((1, 4, 16, 128), data=FAR)]), arr([t((128,))]), FAKE,
                                                         1 << 40, None) == NULL
    x, pos = torch.zeros(1, 1, 4, 64), torch.zeros(4, 1)
    with pytest.raises(cp.CpattnError) as e:
        cp.norm_rotary_backward(x, None, pos, (64,), x, dweights=torch.zeros(64))
    assert e.value.name == "CPATTN_ERR_NULL"
