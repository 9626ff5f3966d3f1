"""Refusals of the rotary-table, q/k norm + rotation, paged cache and paged
attention entry points: the documented codes, before any CUDA call (there is
no device here, so a call that got further would report FRT_ECUDA)."""

import ctypes as C
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A16 = 0x10000  # a fake, 16-byte aligned, never dereferenced address


@pytest.fixture(scope="module")
def frt():
    from fp8_transformer_block_b200 import build
    build.build()
    from fp8_transformer_block_b200 import frt as mod
    return mod


@pytest.fixture(scope="module")
def rt(frt):
    from fp8_transformer_block_b200 import runtime
    return runtime


@pytest.mark.parametrize("name", ["frt_qk_rope_desc", "frt_paged_attn_desc"])
def test_descriptor_layout_matches_header(frt, name):
    src = open(os.path.join(ROOT, "include", "frt.h")).read()
    body = src[src.index("typedef struct " + name):]
    body = re.sub(r"/\*.*?\*/", "", body[:body.index("} " + name + ";")], flags=re.S)
    names = re.findall(r"\**\s*([A-Za-z_][A-Za-z0-9_]*)\s*(?=[,;])", body)
    assert names == [f for f, _ in getattr(frt, name)._fields_]


@pytest.mark.parametrize("change,code", [
    ({}, None), (dict(M=0), 0), (dict(M=-1), -2), (dict(P=-1), -2), (dict(rot=7), -2),
    (dict(rot=0), -2), (dict(theta=0.0), -1), (dict(theta=float("inf")), -1), (dict(scaling=4), -1),
    (dict(scaling=1, factor=0.0), -1), (dict(scaling=1, factor=float("nan")), -1),
    (dict(scaling=2, rot=2), -2), (dict(scaling=3, orig=0.0), -1), (dict(scaling=3, low=32.0), -1),
    (dict(amp=float("nan")), -1), (dict(out=None), -1), (dict(out=A16 + 4), -3)])
def test_table_refusals(frt, change, code):
    a = dict(M=4, rot=64, P=0, theta=1e4, scaling=0, factor=2.0, orig=8192.0, low=1.0, high=32.0,
             amp=1.0, out=A16, stream=None)
    a.update(change)
    if code is not None:
        assert frt.raw_call("frt_build_rope_table_scaled", *a.values()) == code
        assert code == 0 or frt.last_error()


@pytest.mark.parametrize("fmt,ps,hd,want", [
    (0, 16, 64, 16 * 64 * 4), (1, 16, 64, 16 * 64 * 9 // 8), (1, 128, 256, 128 * 256 * 9 // 8),
    (0, 32, 72, 32 * 72 * 4), (1, 32, 72, 0), (0, 8, 64, 0), (0, 48, 64, 0), (0, 2048, 64, 0),
    (1, 16, 8, 0), (0, 16, 264, 0), (2, 16, 64, 0), (0, -16, 64, 0)])
def test_record_bytes(frt, fmt, ps, hd, want):
    assert frt.frt_kv_record_bytes(fmt, ps, hd) == want


def _heads(rt, **kw):
    a = dict(rows=4, hq=4, hkv=2, hd=64, rot=64, layout=1, eps=1e-6, qkv=A16, ld_qkv=512, q_norm=A16,
             k_norm=None, rope=A16, n_pos=100, positions=A16, q_out=A16, ld_q=256, k_out=A16, ld_k=128,
             v_out=A16, ld_v=128, format=1, page_size=16, n_pages=10, pool=A16, slots=A16, k_scale=A16,
             v_scale=A16)
    a.update(kw)
    return rt.qk_rope_desc(**a)


SHARED = [(dict(rows=-1), -2), (dict(hq=-1), -2), (dict(hd=260), -2), (dict(hd=20), -2), (dict(hd=8), -2),
          (dict(rot=24), -2), (dict(rot=80), -2), (dict(rot=-16), -2), (dict(layout=2), -1),
          (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(q_norm=A16 + 8), -3), (dict(rope=None), -1),
          (dict(rope=A16 + 8), -3), (dict(n_pos=0), -2), (dict(positions=None, n_pos=3), -4),
          (dict(positions=A16 + 2), -3), (dict(qkv=None), -1), (dict(qkv=A16 + 8), -3),
          (dict(ld_qkv=516), -3), (dict(ld_q=248), -2), (dict(q_out=A16 + 2), -3), (dict(rows=0), 0)]


@pytest.mark.parametrize("change,code", SHARED + [
    (dict(ld_qkv=376), -2), (dict(q_out=None), -1), (dict(k_out=None), -1), (dict(ld_k=120), -2),
    (dict(hq=0, hkv=0), -2)])
def test_norm_rope_refusals(frt, rt, change, code):
    assert frt.raw_call("frt_qk_norm_rope", C.byref(_heads(rt, **change)), None) == code
    assert code == 0 or frt.last_error()


POOL = [(dict(hkv=0), -2), (dict(format=2), -1), (dict(page_size=24), -2), (dict(page_size=8), -2),
        (dict(n_pages=-1), -2), (dict(pool=None), -1), (dict(slots=None), -1), (dict(pool=A16 + 8), -3),
        (dict(slots=A16 + 4), -3), (dict(k_scale=None), -1), (dict(v_scale=None), -1),
        (dict(v_scale=A16 + 2), -3), (dict(hd=72, rot=64, ld_qkv=1024, ld_q=1024), -2)]


@pytest.mark.parametrize("change,code", SHARED + POOL + [(dict(ld_qkv=504), -2)])
def test_append_refusals(frt, rt, change, code):
    assert frt.raw_call("frt_paged_kv_append", C.byref(_heads(rt, **change)), None) == code


@pytest.mark.parametrize("change,code", POOL + [
    (dict(rows=-1), -2), (dict(rows=0), 0), (dict(k_out=None, v_out=None), -1), (dict(v_out=A16 + 8), -3),
    (dict(ld_v=120), -2), (dict(ld_k=132), -3)])
def test_read_refusals(frt, rt, change, code):
    assert frt.raw_call("frt_paged_kv_read", C.byref(_heads(rt, **change)), None) == code


@pytest.mark.parametrize("change,code", [
    (dict(hd=96), -2), (dict(hq=7), -2), (dict(hkv=0), -2), (dict(n_seqs=-1), -2), (dict(rows=-1), -2),
    (dict(max_q=-1), -2), (dict(page_size=20), -2), (dict(max_pages=-1), -2), (dict(n_pages=-1), -2),
    (dict(max_pages=1 << 30), -2), (dict(window=-1), -1), (dict(window=4, causal=0), -1), (dict(q=None), -1),
    (dict(out=None), -1), (dict(kv_len=None), -1), (dict(k_scale=None), -1), (dict(pool=None), -1),
    (dict(page_table=None), -1), (dict(q=A16 + 8), -3), (dict(pool=A16 + 8), -3), (dict(ld_q=516), -3),
    (dict(ld_q=504), -2), (dict(ld_out=504), -2), (dict(cu_rows=A16 + 2), -3), (dict(lse=A16 + 1), -3),
    (dict(workspace=None), -1), (dict(workspace=A16 + 4), -3), (dict(workspace_bytes=16), -4),
    (dict(sm_scale=float("nan")), -1), (dict(sm_scale=float("inf")), -1),
    (dict(n_seqs=0), 0), (dict(rows=0), 0), (dict(max_q=0), 0)])
def test_attention_refusals(frt, rt, change, code):
    a = dict(n_seqs=3, rows=3, max_q=1, hq=8, hkv=2, hd=64, page_size=16, max_pages=8, n_pages=24, causal=1,
             window=0, sm_scale=0.125, q=A16, ld_q=512, pool=A16, page_table=A16, cu_rows=A16, kv_len=A16,
             k_scale=A16, v_scale=A16, out=A16, ld_out=512, lse=None, workspace=A16,
             workspace_bytes=1 << 30)
    a.update(change)
    assert frt.raw_call("frt_paged_attention_fp4", C.byref(rt.paged_attn_desc(**a)), None) == code
    assert code == 0 or frt.last_error()


def test_null_descriptors(frt):
    for name in ("frt_qk_norm_rope", "frt_paged_kv_append", "frt_paged_kv_read", "frt_paged_attention_fp4"):
        assert frt.raw_call(name, None, None) == frt.FRT_EINVAL


def test_workspace_size(frt):
    """Of the heads and the rows alone, and 0 for what the call refuses."""
    assert frt.frt_paged_attention_workspace_size(4, 1, 8, 1, 128) > 0
    assert frt.frt_paged_attention_workspace_size(4, 1, 8, 3, 128) == 0
    assert frt.frt_paged_attention_workspace_size(4, 1, 8, 1, 96) == 0
    assert frt.frt_paged_attention_workspace_size(-1, 1, 8, 1, 64) == 0


@pytest.mark.parametrize("unused", [dict(hq=-1), dict(hq=1 << 20), dict(rot=7, layout=9, eps=-1.0, n_pos=-1, rope=A16 + 2),
                                    dict(qkv=None, ld_qkv=3, q_out=A16 + 2, ld_q=1, q_norm=A16 + 2)])
def test_read_does_not_look_at_other_fields(frt, rt, unused):
    """frt_paged_kv_read uses rows, hkv, hd, k_out, v_out and the page fields
    only: nothing else is a reason to refuse (rows = 0 ends ahead of the
    device)."""
    assert frt.raw_call("frt_paged_kv_read", C.byref(_heads(rt, rows=0, **unused)), None) == 0
    assert frt.raw_call("frt_paged_kv_read", C.byref(_heads(rt, page_size=24, **unused)), None) == -2
