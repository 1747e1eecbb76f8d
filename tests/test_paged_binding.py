"""Refusals of the paged entry points, at the C entries and in the binding: bad sizes,
types, strides and alignments return before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

import sparse_mla_decoding_b200 as smla

FAKE = ctypes.c_void_p(0x10000)      # never dereferenced: the calls fail validation first


def cache(**kw):
    f = dict(k_cache=0x10000, v_cache=0x10000, k_scale=0x10000, v_scale=0x10000, num_blocks=4,
             k_block_stride=2 * 64 * 128, v_block_stride=2 * 64 * 128, k_scale_stride=2, v_scale_stride=2, h_kv=2,
             head_dim=128, format=0)
    f.update(kw)
    return smla._Q8Cache(**f)


BAD_CACHES = [(dict(head_dim=96), 2), (dict(format=2), 2), (dict(format=-1), 2), (dict(h_kv=0), 1),
              (dict(k_cache=None), 1), (dict(v_scale=None), 1), (dict(num_blocks=0), 1), (dict(num_blocks=1 << 26), 1),
              (dict(k_block_stride=2 * 64 * 128 - 16), 1), (dict(v_block_stride=2 * 64 * 128 + 8), 1),
              (dict(k_scale_stride=1), 1), (dict(k_cache=0x10008), 1), (dict(v_scale=0x10002), 1),
              (dict(h_kv=1 << 20), 1)]


def write_args(**kw):
    a = dict(k=FAKE, v=FAKE, kts=256, khs=128, vts=256, vhs=128, total=10, cache=cache(), table=FAKE, cols=4, batch=2,
             lens=FAKE, new=FAKE, cu=FAKE, status=None, stream=None)
    a.update(kw)
    a["cache"] = ctypes.byref(a["cache"]) if a["cache"] is not None else None
    return list(a.values())


def attend_args(**kw):
    a = dict(q=FAKE, qts=1024, qhs=128, total=6, h_q=8, cache=cache(), table=FAKE, cols=4, batch=3, lens=FAKE, cu=FAKE,
             s_q=0, hint=2, causal=1, scale=-1.0, cap=0.0, slopes=None, prefix=None, docs=None, o=FAKE, lse=FAKE,
             ws=FAKE, ws_bytes=1 << 40, status=None, stream=None)
    a.update(kw)
    a["cache"] = ctypes.byref(a["cache"]) if a["cache"] is not None else None
    return list(a.values())


def table_args(**kw):
    a = dict(table=FAKE, cols=4, lens=FAKE, new=FAKE, batch=2, free=FAKE, cap=5, num_free=FAKE, most=10, slots=FAKE,
             cu=FAKE, out=ctypes.c_void_p(0x20000), left=ctypes.c_void_p(0x30000), stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_bad_caches(change, status):
    L = smla.lib()
    assert L.smla_quantize_kv_blocks(*write_args(cache=cache(**change))) == status
    assert L.smla_gqa_attention_with_kvcache(*attend_args(cache=cache(**change))) == status


@pytest.mark.parametrize("change", [dict(cache=None), dict(k=None), dict(v=None), dict(table=None), dict(lens=None),
                                    dict(new=None), dict(cu=None), dict(total=-1), dict(total=1 << 31), dict(cols=0),
                                    dict(batch=-1), dict(kts=257), dict(vhs=4), dict(khs=-8),
                                    dict(k=ctypes.c_void_p(0x10008)), dict(cache=cache(h_kv=65536, k_scale_stride=65536,
                                    v_scale_stride=65536, head_dim=64, k_block_stride=1 << 28, v_block_stride=1 << 28))])
def test_bad_writes(change):
    assert smla.lib().smla_quantize_kv_blocks(*write_args(**change)) == 1


@pytest.mark.parametrize("change", [dict(cache=None), dict(q=None), dict(table=None), dict(lens=None), dict(o=None),
                                    dict(lse=None), dict(ws=None), dict(h_q=7), dict(h_q=0), dict(batch=-1),
                                    dict(cols=0), dict(total=-1), dict(total=1 << 31), dict(total=1 << 30, h_q=8),
                                    dict(causal=2), dict(hint=-1), dict(cu=None), dict(cu=None, s_q=3),
                                    dict(cap=-1.0), dict(cap=float("nan")), dict(cap=float("inf")), dict(cap=1e-30), dict(cap=1e30),
                                    dict(scale=1e-40),
                                    dict(scale=float("inf")), dict(prefix=FAKE, causal=0), dict(qts=1025),
                                    dict(qhs=-8), dict(q=ctypes.c_void_p(0x10002)), dict(o=ctypes.c_void_p(0x10008)),
                                    dict(ws=ctypes.c_void_p(0x10010)), dict(docs=ctypes.c_void_p(0x10004))])
def test_bad_attention_calls(change):
    assert smla.lib().smla_gqa_attention_with_kvcache(*attend_args(**change)) == 1


@pytest.mark.parametrize("change", [dict(batch=-1), dict(cols=0), dict(cap=-1), dict(most=-1), dict(most=1 << 31),
                                    dict(num_free=None), dict(cu=None), dict(left=None), dict(slots=None),
                                    dict(free=None), dict(table=None), dict(lens=None), dict(new=None),
                                    dict(out=None), dict(left=FAKE, num_free=FAKE), dict(out=FAKE)])
def test_bad_table_calls(change):
    assert smla.lib().smla_extend_block_table(*table_args(**change)) == 1


def test_empty_calls_do_nothing():
    L = smla.lib()
    assert L.smla_quantize_kv_blocks(*write_args(total=0, k=None, v=None)) == 0
    assert L.smla_quantize_kv_blocks(*write_args(batch=0)) == 0
    assert L.smla_gqa_attention_with_kvcache(*attend_args(total=0, q=None, o=None, lse=None)) == 0
    assert L.smla_gqa_attention_with_kvcache(*attend_args(batch=0)) == 0
    assert L.smla_gqa_workspace_bytes(96, 0) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    k = torch.zeros(4, 2, 64, 128, dtype=torch.int8)
    s = torch.zeros(4, 2)
    i = torch.zeros(1, dtype=torch.int32)
    q = torch.zeros(1, 1, 8, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="k_cache"):
        smla.gqa_attention_with_kvcache(q, k, k, s, s, i.view(1, 1), i)
    with pytest.raises(ValueError, match="k_cache"):
        smla.quantize_kv_blocks(q[0], q[0], k, k, s, s, i.view(1, 1), i, i, i)
    with pytest.raises(ValueError, match="block_table"):
        smla.extend_block_table(i.view(1, 1), i, i, i, i, 1)
    assert smla.paged_status.__doc__ and smla._paged_words == {}
