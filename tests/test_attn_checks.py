"""The attention operators' refusals: bad arguments return before anything is
launched (no GPU needed)."""
import ctypes
import os
import re

import pytest
import torch

import bit_dequant_expert_b200 as m

FAKE = 0x7F0000000000   # 256-byte aligned, never dereferenced: every case fails validation first
INV, UNS, WS = m.MOE_ERR_INVALID_ARG, m.MOE_ERR_UNSUPPORTED, m.MOE_ERR_WORKSPACE
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def cfg(**kw):
    return m.attn_config(**{**dict(q_heads=16, kv_heads=2, head_dim=128, page_size=64, cache_type=1), **kw})


BAD_CONFIGS = [(dict(q_heads=0), INV), (dict(kv_heads=0), INV), (dict(q_heads=15), INV), (dict(cache_type=2), INV),
               (dict(head_dim=96), UNS), (dict(head_dim=512), UNS), (dict(page_size=8), UNS), (dict(page_size=48), UNS),
               (dict(q_heads=130, kv_heads=2), UNS), (dict(q_heads=512, kv_heads=64), UNS)]


def prepare(c=None, **kw):
    a = dict(T=4, qkv=FAKE, qkv_stride=20 * 128, q_weight=FAKE, k_weight=FAKE, eps=1e-6, inv_freq=FAKE, rot_dim=128,
             rope_layout=0, rope_scale=1.0, positions=FAKE, slots=FAKE, num_pages=4, k_cache=FAKE, v_cache=FAKE,
             k_scale=FAKE, v_scale=FAKE, q_out=FAKE, k_out=None)
    a.update(kw)
    return m.attn_qkv_prepare(c or cfg(), *a.values(), stream=0, raise_on_error=False)


def read(c=None, **kw):
    a = dict(B=2, total=8, page_table=FAKE, page_table_stride=3, cu_lens=FAKE, num_pages=4, k_cache=FAKE, v_cache=FAKE,
             k_scale=FAKE, v_scale=FAKE, k_out=FAKE, v_out=FAKE)
    a.update(kw)
    return m.attn_kv_read(c or cfg(), *a.values(), stream=0, raise_on_error=False)


def prefill(c=None, **kw):
    a = dict(B=2, total_q=8, total_k=8, cu_q=FAKE, cu_k=FAKE, q=FAKE, q_stride=16 * 128, k=FAKE, k_stride=256, v=FAKE,
             v_stride=256, scale=0.1, causal=1, out=FAKE, lse=None)
    a.update(kw)
    return m.attn_prefill(c or cfg(), *a.values(), stream=0, raise_on_error=False)


def decode(c=None, **kw):
    a = dict(B=2, nq=1, max_len=100, q=FAKE, q_stride=16 * 128, page_table=FAKE, page_table_stride=2, seq_lens=FAKE,
             num_pages=4, k_cache=FAKE, v_cache=FAKE, k_scale=FAKE, v_scale=FAKE, scale=0.1, out=FAKE, lse=None,
             ws=FAKE, ws_bytes=1 << 40)
    a.update(kw)
    return m.attn_decode(c or cfg(), *a.values(), stream=0, raise_on_error=False)


def test_header_is_exported():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "attn_b200.h")).read(), flags=re.S)
    names = set(re.findall(r"^(?:int32_t|size_t) (attn_\w+)\(", text, flags=re.M))
    assert names == {"attn_qkv_prepare", "attn_kv_read", "attn_prefill", "attn_decode_workspace_size", "attn_decode"}
    lib = ctypes.CDLL(m.LIB_PATH)
    assert all(hasattr(lib, n) for n in names) and names <= set(m.EXPORTED)


@pytest.mark.parametrize("bad,status", BAD_CONFIGS)
def test_bad_configs(bad, status):
    c = cfg(**bad)
    for call in (prepare, read, prefill, decode):
        assert call(c) == status
    assert m.attn_decode_workspace_size(c, 1, 1, 100) == 0


@pytest.mark.parametrize("bad,status", [
    (dict(T=0), INV), (dict(T=-1), INV), (dict(qkv=None), INV), (dict(qkv=FAKE + 8), INV), (dict(q_out=None), INV),
    (dict(q_out=FAKE + 4), INV), (dict(k_out=FAKE + 2), INV), (dict(qkv_stride=20 * 128 - 8), INV),
    (dict(qkv_stride=20 * 128 + 4), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(eps=float("inf")), INV), (dict(rope_scale=float("nan")), INV), (dict(rope_layout=2), INV),
    (dict(rot_dim=136), UNS), (dict(rot_dim=8), UNS), (dict(rot_dim=-16), UNS), (dict(inv_freq=None), INV),
    (dict(positions=None), INV), (dict(positions=FAKE + 2), INV), (dict(slots=FAKE + 1), INV), (dict(num_pages=0), INV),
    (dict(k_cache=None), INV), (dict(v_cache=FAKE + 8), INV), (dict(k_scale=None), INV), (dict(v_scale=FAKE + 4), INV),
    (dict(q_weight=FAKE + 2), INV), (dict(num_pages=1 << 26), UNS)])
def test_prepare_refuses(bad, status):
    assert prepare(**bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(B=0), INV), (dict(total=-1), INV), (dict(page_table=None), INV), (dict(page_table_stride=0), INV),
    (dict(cu_lens=None), INV), (dict(k_out=None), INV), (dict(v_out=FAKE + 8), INV), (dict(num_pages=0), INV),
    (dict(v_cache=None), INV), (dict(v_scale=None), INV), (dict(total=0), m.MOE_OK)])
def test_read_refuses(bad, status):
    assert read(**bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(B=0), INV), (dict(total_q=0), INV), (dict(total_k=-1), INV), (dict(cu_q=None), INV), (dict(cu_k=None), INV),
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=FAKE + 8), INV), (dict(q_stride=2040), INV),
    (dict(k_stride=260), INV), (dict(v_stride=248), INV), (dict(scale=float("inf")), INV), (dict(causal=2), INV),
    (dict(out=None), INV), (dict(lse=FAKE + 2), INV), (dict(total_q=1 << 26), UNS), (dict(total_k=1 << 26), UNS),
    (dict(B=65536), UNS)])
def test_prefill_refuses(bad, status):
    assert prefill(**bad) == status


@pytest.mark.parametrize("bad,status", [
    (dict(B=0), INV), (dict(nq=0), INV), (dict(nq=9), UNS), (dict(B=65536), UNS), (dict(max_len=0), INV),
    (dict(q=None), INV), (dict(q=FAKE + 8), INV), (dict(q_stride=2040), INV), (dict(page_table=None), INV),
    (dict(page_table_stride=1), INV), (dict(seq_lens=None), INV), (dict(scale=float("nan")), INV),
    (dict(out=None), INV), (dict(k_scale=None), INV), (dict(ws=None), WS), (dict(ws=FAKE + 16), WS),
    (dict(ws_bytes=0), WS)])
def test_decode_refuses(bad, status):
    assert decode(**bad) == status


def test_counts_and_strides_past_the_limits_are_refused():
    far = (1 << 31) + 8
    assert read(page_table_stride=far) == INV and decode(page_table_stride=far) == INV
    assert decode(max_len=(1 << 30) + 1, page_table_stride=1 << 25) == UNS
    assert decode(B=65535, max_len=1 << 30, page_table_stride=1 << 25) == UNS
    c = cfg()
    assert m.attn_decode_workspace_size(c, 1, 1, 1 << 30) > 0
    assert m.attn_decode_workspace_size(c, 1, 1, (1 << 30) + 1) == 0
    assert m.attn_decode_workspace_size(c, 65535, 1, 1 << 30) == 0


def test_workspace_size():
    c = cfg()
    assert m.attn_decode_workspace_size(c, 1, 1, 1) > 0
    assert m.attn_decode_workspace_size(c, 0, 1, 1) == 0 and m.attn_decode_workspace_size(c, 1, 9, 1) == 0
    assert m.attn_decode_workspace_size(c, 1, 1, 0) == 0 and m.attn_decode_workspace_size(c, 65536, 1, 1) == 0


def test_binding_refuses_tensors_the_library_cannot_read():
    t = torch.zeros(4, 20 * 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="qkv is on cpu"):
        prepare(qkv=t)
    with pytest.raises(ValueError, match="q is on cpu"):
        decode(q=t)
    with pytest.raises(ValueError, match="cu_q is on cpu"):
        prefill(cu_q=torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="k_out is on cpu"):
        read(k_out=t)


def test_layer_refuses_bad_shapes():
    with pytest.raises(ValueError, match="unsupported"):
        m.AttentionLayer(16, 2, 96, 4, device="cuda:0")
    with pytest.raises(ValueError, match="unsupported"):
        m.AttentionLayer(16, 3, 128, 4, device="cuda:0")
    with pytest.raises(ValueError, match="num_pages"):
        m.AttentionLayer(16, 2, 128, 0, device="cuda:0")
    with pytest.raises(ValueError, match="q_weight"):
        m.AttentionLayer(16, 2, 128, 4, q_weight=torch.ones(64), device="cuda:0")
    with pytest.raises(ValueError, match="inv_freq"):
        m.AttentionLayer(16, 2, 128, 4, inv_freq=torch.ones(12), device="cuda:0")


@pytest.mark.parametrize("device", ["cpu", "meta", torch.device("cpu")])
def test_layer_refuses_other_devices(device):
    with pytest.raises(ValueError, match="runs on a GPU"):
        m.AttentionLayer(16, 2, 128, 4, device=device)


def test_read_refuses_more_rows_than_it_can_number():
    for total in (0x7FFFFF01, 0x7FFFFF81, 0x7FFFFFFF):
        assert read(total=total) == UNS


def test_scales_that_overflow_in_log2_units_are_refused():
    for scale in (2.4e38, -3e38):
        assert prefill(scale=scale) == INV and decode(scale=scale) == INV
