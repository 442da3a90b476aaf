"""The 4-bit row's definition as the tests hold it, against facts that do not come from it, and the calls that the
library refuses without a GPU."""
import ctypes

import numpy as np
import pytest

import decode_kv_cache_paged_b200 as kvc
import rows4


def test_values_are_within_half_a_step():
    rng = np.random.default_rng(1)
    x = rng.normal(size=(50, 128)).astype(np.float32)
    x = (x.view(np.uint32) & 0xFFFF0000).view(np.float32).astype(np.float64)
    step, lo, codes = rows4.code_rows(x)
    v = rows4.row_values(x)
    assert np.all(np.abs(v - x).reshape(50, 4, 32) <= step[..., None] / 2)
    g = x.reshape(50, 4, 32)
    assert np.array_equal(lo, g.min(-1))
    # the step covers the range, and is at most one 1/8 wider than it has to be (four significant bits)
    need = (g.max(-1) - lo) / 15
    assert np.all(step >= need) and np.all(step <= need * (1 + 1 / 8))
    assert np.all(step * 2.0 ** (3 - np.floor(np.log2(step))) % 1 == 0)


def test_ties_go_to_even_codes():
    x = np.zeros((1, 64))
    x[0, :4] = [0.0, 15.0, 2.5, 3.5]  # step 1: 2.5 -> 2, 3.5 -> 4
    assert rows4.row_values(x)[0, :4].tolist() == [0.0, 15.0, 2.0, 4.0]


def test_constant_and_broken_groups():
    x = np.full((1, 64), -3.0)
    x[0, 16] = np.inf
    x[0, 40] = np.nan
    v = rows4.row_values(x)[0].reshape(4, 16)
    assert np.all(v[0] == -3.0) and np.all(np.isnan(v[1])) and np.all(np.isnan(v[2])) and np.all(v[3] == -3.0)


def test_attention_round_reference():
    w = np.array([9, 9, 5, 7, 7, 1, np.nan, 0.5])
    pos = np.arange(8)
    # prompt 2, budget 5: the newest position, then 7 and 7 (lower position first)
    assert rows4.attention_round(w, pos, 2, 5, 1, 8).tolist() == [0, 1, 3, 4, 7]
    assert rows4.attention_round(w, pos, 2, 4, 9, 8).tolist() == [0, 1, 6, 7]
    assert rows4.compacted(np.array([0, 3, 5, 7]), 4, True).tolist() == [0, 5, 7, 3]


def _cfg(**kw):
    base = dict(num_requests=4, num_layers=2, num_kv_heads=8, num_q_heads=32, head_dim=128, page_size=16,
                dtype=kvc.KVC_INT4, num_beacons=0, query_window=0, max_seq_len=2112, num_pages=600)
    base.update(kw)
    return kvc.kvc_config(**base)


def test_workspace_of_a_4bit_context():
    n4 = kvc.kvc_workspace_bytes(ctypes.byref(_cfg(query_window=8)))
    n16 = kvc.kvc_workspace_bytes(ctypes.byref(_cfg(query_window=8, dtype=kvc.KVC_BF16)))
    assert n4 == n16 > 0  # queries are kept in bf16 either way


@pytest.mark.parametrize("bad", [dict(head_dim=96), dict(head_dim=256), dict(head_dim=32),
                                 dict(num_beacons=64, query_window=64), dict(dtype=3), dict(dtype=-1)])
def test_4bit_configs_refused(bad):
    assert kvc.kvc_workspace_bytes(ctypes.byref(_cfg(**bad))) == 0
    h = ctypes.c_void_p()
    assert kvc.kvc_create(ctypes.byref(_cfg(**bad)), None, None, None, 0, None, ctypes.byref(h)) == kvc.KVC_ERR_INVALID_ARG
    assert kvc.kvc_last_error(None) and not h


def test_null_handles():
    assert kvc.kvc_bind_weights(None, None, 0) == kvc.KVC_ERR_INVALID_ARG
    assert kvc.kvc_decode_attention_ex(None, 0, 1, None, 0.0, None, None, None, None) == kvc.KVC_ERR_INVALID_ARG


def test_dtype_names():
    import torch
    assert kvc._dtype_code("int4") == kvc.KVC_INT4 and kvc._dtype_code(torch.bfloat16) == kvc.KVC_BF16
    with pytest.raises(ValueError):
        kvc._dtype_code(torch.float16)
