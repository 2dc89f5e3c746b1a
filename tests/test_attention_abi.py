"""Host-side validation of the softmax-attention operators: the C ABI and the
binding refuse bad arguments before any launch.  No GPU: no call here reaches
one."""
import ctypes
import os
import subprocess

import pytest
import torch

import attnref as ref
import linear_attention_recurrent_int8_b200 as lq

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
OK, INVALID, UNSUPPORTED, MISALIGNED = lq.LQ_OK, lq.LQ_ERR_INVALID_ARGUMENT, lq.LQ_ERR_UNSUPPORTED, lq.LQ_ERR_MISALIGNED
PTR = 1 << 20  # an aligned address that is never followed


def cfg_c(**kw):
    return lq.AttnConfig(**{**dict(q_heads=8, kv_heads=2, head_dim=128), **kw}).c()


def cache_c(**kw):
    d = dict(k_pages=PTR, v_pages=PTR, block_table=PTR, batch=4, num_pages=10, page_size=64, max_pages=8)
    return lq.LqKvCache(*{**d, **kw}.values())


def norm_call(cfg, **kw):
    d = dict(q=PTR, q_stride=1024, k=PTR, k_stride=256, qw=None, kw=None, positions=None, table=None, table_len=0,
             tokens=0x7fff0000, q_out=PTR, k_out=PTR, stream=None)
    return lq.load_library().lq_qk_norm_rotate(ctypes.byref(cfg), *{**d, **kw}.values())


def append_call(cfg, cache, **kw):
    d = dict(pos=PTR, cu=None, tokens=8, q=PTR, q_stride=1024, k=PTR, k_stride=256, v=PTR, v_stride=256, qw=None, kw=None,
             table=None, table_len=0, q_out=PTR, stream=None)
    return lq.load_library().lq_kv_append(ctypes.byref(cfg), ctypes.byref(cache), *{**d, **kw}.values())


def decode_call(cfg, cache, **kw):
    d = dict(pos=PTR, q=PTR, o=PTR, ws=PTR, ws_bytes=0, stream=None)
    return lq.load_library().lq_attn_decode(ctypes.byref(cfg), ctypes.byref(cache), *{**d, **kw}.values())


def prefill_call(cfg, cache, **kw):
    d = dict(pos=PTR, cu=None, tokens=8, q=PTR, o=PTR, stream=None)
    return lq.load_library().lq_attn_prefill(ctypes.byref(cfg), ctypes.byref(cache), *{**d, **kw}.values())


BAD_CONFIGS = [
    (dict(q_heads=7), INVALID), (dict(q_heads=0), INVALID), (dict(kv_heads=0), INVALID),
    (dict(q_heads=4098), INVALID), (dict(head_dim=0), INVALID), (dict(head_dim=96), UNSUPPORTED),
    (dict(io_dtype=2), INVALID), (dict(norm=3), INVALID), (dict(norm=1, eps=0.0), INVALID),
    (dict(norm=1, eps=float("nan")), INVALID), (dict(norm=2, eps=float("inf")), INVALID),
    (dict(rot_dim=8), INVALID), (dict(rot_dim=-16), INVALID), (dict(rot_dim=144), INVALID),
    (dict(rot_pairs=2), INVALID), (dict(window=-1), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(softcap=-1.0), INVALID), (dict(softcap=float("nan")), INVALID),
]


@pytest.mark.parametrize("change,status", BAD_CONFIGS)
def test_configurations_are_refused(change, status):
    c = cfg_c(**change)
    assert norm_call(c) == status
    assert append_call(c, cache_c()) == status
    assert decode_call(c, cache_c()) == status
    assert prefill_call(c, cache_c()) == status
    assert lq.load_library().lq_attn_workspace_bytes(ctypes.byref(c), 4) == -1


BAD_CACHES = [
    (dict(k_pages=None), INVALID), (dict(v_pages=None), INVALID), (dict(block_table=None), INVALID),
    (dict(batch=0), INVALID), (dict(batch=4097), UNSUPPORTED), (dict(num_pages=0), INVALID),
    (dict(num_pages=1 << 30), INVALID), (dict(page_size=0), INVALID), (dict(page_size=8), UNSUPPORTED),
    (dict(page_size=48), UNSUPPORTED), (dict(page_size=512), UNSUPPORTED), (dict(max_pages=0), INVALID),
    (dict(max_pages=1 << 24), INVALID), (dict(k_pages=PTR + 8), MISALIGNED), (dict(v_pages=PTR + 2), MISALIGNED),
    (dict(block_table=PTR + 1), MISALIGNED),
]


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_caches_are_refused(change, status):
    for call in (append_call, decode_call, prefill_call):
        assert call(cfg_c(), cache_c(**change)) == status


def test_norm_arguments_are_refused():
    c, rot = cfg_c(), cfg_c(rot_dim=64)
    assert norm_call(c, tokens=0) == OK
    for change in (dict(tokens=-1), dict(q=None), dict(q_out=None), dict(k=None), dict(k_out=None),
                   dict(q_stride=1023), dict(k_stride=255), dict(q_stride=1 << 41), dict(qw=PTR), dict(kw=PTR),
                   dict(table=PTR, table_len=4)):
        assert norm_call(c, **change) == INVALID, change
    for change in (dict(q=PTR + 8), dict(k=PTR + 2), dict(q_out=PTR + 8), dict(k_out=PTR + 4), dict(q_stride=1028),
                   dict(positions=PTR + 2)):
        assert norm_call(c, **change) == MISALIGNED, change
    assert norm_call(rot, positions=PTR) == INVALID
    assert norm_call(rot, table=PTR, table_len=4) == INVALID
    assert norm_call(rot, positions=PTR, table=PTR, table_len=0) == INVALID
    assert norm_call(rot, positions=PTR, table=PTR + 4, table_len=9) == MISALIGNED
    assert norm_call(cfg_c(norm=2), qw=PTR + 4) == MISALIGNED


def test_append_arguments_are_refused():
    c, k = cfg_c(), cache_c()
    assert append_call(c, k, tokens=0) == OK
    for change in (dict(tokens=-4), dict(tokens=9), dict(pos=None), dict(q=None), dict(q_out=None), dict(k=None),
                   dict(v=None), dict(v_stride=128), dict(k_stride=-256), dict(kw=PTR), dict(table=PTR, table_len=3)):
        assert append_call(c, k, **change) == INVALID, change
    for change in (dict(pos=PTR + 2), dict(cu=PTR + 1), dict(q=PTR + 8), dict(v=PTR + 8), dict(v_stride=260),
                   dict(q_out=PTR + 2)):
        assert append_call(c, k, **change) == MISALIGNED, change
    assert append_call(cfg_c(rot_dim=64), k) == INVALID


def test_attention_arguments_are_refused():
    c, k = cfg_c(), cache_c()
    for change in (dict(pos=None), dict(q=None), dict(o=None), dict(ws=None)):
        assert decode_call(c, k, **change) == INVALID, change
    for change in (dict(pos=PTR + 1), dict(q=PTR + 2), dict(o=PTR + 8), dict(ws=PTR + 4)):
        assert decode_call(c, k, **change) == MISALIGNED, change
    # more tokens than the line of tiles counts
    assert decode_call(c, cache_c(batch=4096, max_pages=1 << 18, page_size=16)) == UNSUPPORTED
    assert prefill_call(c, k, tokens=0) == OK
    for change in (dict(pos=None), dict(q=None), dict(o=None), dict(tokens=-8), dict(tokens=3)):
        assert prefill_call(c, k, **change) == INVALID, change
    for change in (dict(pos=PTR + 1), dict(cu=PTR + 3), dict(q=PTR + 2), dict(o=PTR + 8)):
        assert prefill_call(c, k, **change) == MISALIGNED, change
    lib = lq.load_library()
    assert lib.lq_attn_workspace_bytes(ctypes.byref(c), 0) == -1
    assert lib.lq_attn_workspace_bytes(ctypes.byref(c), 4097) == -1
    assert lib.lq_attn_workspace_bytes(None, 1) == -1


def test_structs_match_the_header_layout(tmp_path):
    src = tmp_path / "layout.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "lq.h"\nint main(void) {\n'
                   + "".join(f'printf("{s} {f} %zu\\n", offsetof({s}, {f}));\n'
                             for s, t in (("lq_attn_config", lq.LqAttnConfig), ("lq_kv_cache", lq.LqKvCache))
                             for f, _ in t._fields_)
                   + 'printf("%zu %zu\\n", sizeof(lq_attn_config), sizeof(lq_kv_cache));\n'
                     'printf("%d %d %d %d %d %u\\n", LQ_NORM_NONE, LQ_NORM_L2, LQ_NORM_RMS, LQ_ROT_HALVES, '
                     'LQ_ROT_ADJACENT, LQ_DEVERR_BAD_PAGE);\nreturn 0; }\n')
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I" + os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split("\n")
    want = [f"{s} {f} {getattr(t, f).offset}"
            for s, t in (("lq_attn_config", lq.LqAttnConfig), ("lq_kv_cache", lq.LqKvCache)) for f, _ in t._fields_]
    assert lines[:len(want)] == want
    assert lines[len(want)] == f"{ctypes.sizeof(lq.LqAttnConfig)} {ctypes.sizeof(lq.LqKvCache)}"
    assert lines[len(want) + 1] == "0 1 2 0 1 4"


# ------------------------------------------------------------------ the binding

@pytest.fixture
def no_library(monkeypatch):
    def _refuse(*a, **k):
        raise AssertionError("the library was called")
    monkeypatch.setattr(lq, "load_library", _refuse)


def zeros(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def test_cache_object_checks_its_tensors():
    cfg = lq.AttnConfig(4, 2, 64)
    k, table = zeros(9, 2, 16, 64), zeros(3, 5, dtype=torch.int32)
    c = lq.KvCache(cfg, k, k.clone(), table)
    assert (c.batch, c.max_pages, c.num_pages, c.page_size) == (3, 5, 9, 16)
    with pytest.raises(TypeError, match="k_pages: dtype"):
        lq.KvCache(cfg, k.float(), k, table)
    with pytest.raises(ValueError, match="v_pages: shape"):
        lq.KvCache(cfg, k, zeros(9, 2, 32, 64), table)
    with pytest.raises(ValueError, match="k_pages: shape"):
        lq.KvCache(cfg, zeros(9, 4, 16, 64), k, table)
    with pytest.raises(ValueError, match="not contiguous"):
        lq.KvCache(cfg, zeros(9, 16, 2, 64).transpose(1, 2), k, table)
    with pytest.raises(TypeError, match="block_table: dtype"):
        lq.KvCache(cfg, k, k, table.long())
    with pytest.raises(ValueError, match="block_table: shape"):
        lq.KvCache(cfg, k, k, table.view(-1))
    with pytest.raises(AttributeError):
        c.k_pages = k  # the C struct holds the pointers


def test_binding_rejects_bad_tensors_before_the_library(no_library):
    cfg = lq.AttnConfig(4, 2, 64, rot_dim=32, norm=lq.LQ_NORM_RMS)
    kp, table = zeros(9, 2, 16, 64), zeros(3, 5, dtype=torch.int32)
    cache = lq.KvCache(cfg, kp, kp.clone(), table)
    q, k = zeros(6, 4, 64), zeros(6, 2, 64)
    pos, cs, w = zeros(6, dtype=torch.int32), zeros(10, 32, dtype=torch.float32), zeros(64, dtype=torch.float32)

    def norm(**kw):
        d = dict(q=q, k=k, q_weight=w, k_weight=w, positions=pos, cos_sin=cs, q_out=q.clone(), k_out=k.clone())
        lq.lq_qk_norm_rotate(cfg, **{**d, **kw})

    for kw, kind, match in [
            (dict(q=q.float()), TypeError, "q: dtype"), (dict(q=zeros(6, 5, 64)), ValueError, "q: shape"),
            (dict(k=zeros(5, 2, 64)), ValueError, "k: 5 tokens"), (dict(k=None), ValueError, "k and k_out"),
            (dict(q=zeros(6, 64, 4).transpose(1, 2)), ValueError, "not contiguous"),
            (dict(q=zeros(2, 5, 4, 64)[:, :3]), ValueError, "one stride"),
            (dict(q_out=zeros(6, 4, 128)[..., :64]), ValueError, "q_out: not contiguous"),
            (dict(k_out=zeros(6, 4, 64)), ValueError, "k_out: shape"),
            (dict(q_weight=w[:32]), ValueError, "q_weight"), (dict(k_weight=w.double()), TypeError, "k_weight"),
            (dict(positions=pos[:5]), ValueError, "positions"), (dict(positions=pos.long()), TypeError, "positions"),
            (dict(cos_sin=cs[:, :16]), ValueError, "cos_sin"), (dict(cos_sin=zeros(10, 64, dtype=torch.float32)), ValueError, "cos_sin"),
            (dict(), ValueError, "CUDA")]:
        with pytest.raises(kind, match=match):
            norm(**kw)

    start = zeros(3, dtype=torch.int32)
    cu = zeros(4, dtype=torch.int32)

    def append(**kw):
        d = dict(cache=cache, pos=start, cu_tokens=cu, q=q, k=k, v=k, q_weight=w, k_weight=w, cos_sin=cs, q_out=q.clone())
        lq.lq_kv_append(cfg, **{**d, **kw})

    other = lq.AttnConfig(4, 2, 64, io_dtype=lq.LQ_F32)
    wrong = lq.KvCache(other, kp.float(), kp.float(), table)
    for kw, kind, match in [
            (dict(cache=wrong), ValueError, "cache: made for"), (dict(cache=kp), TypeError, "KvCache"),
            (dict(v=zeros(5, 2, 64)), ValueError, "v: 5 tokens"), (dict(q=None), ValueError, "q and q_out"),
            (dict(pos=start[:2]), ValueError, "pos"), (dict(cu_tokens=start), ValueError, "cu_tokens"),
            (dict(cu_tokens=cu.long()), TypeError, "cu_tokens"),
            (dict(cu_tokens=None, q=zeros(5, 4, 64), k=zeros(5, 2, 64), v=zeros(5, 2, 64), q_out=zeros(5, 4, 64)),
             ValueError, "need cu_tokens"),
            (dict(), ValueError, "CUDA")]:
        with pytest.raises(kind, match=match):
            append(**kw)

    q3 = zeros(3, 4, 64)
    for args, kind, match in [
            ((cache, start, zeros(4, 4, 64), q3), ValueError, "q: shape"), ((cache, start, q3, q3.float()), TypeError, "o: dtype"),
            ((cache, start.long(), q3, q3), TypeError, "pos"), ((wrong, start, q3, q3), ValueError, "cache"),
            ((cache, start, q3, q3, "mine"), ValueError, "CUDA|workspace"), ((cache, start, q3, q3), ValueError, "CUDA")]:
        with pytest.raises(kind, match=match):
            lq.lq_attn_decode(cfg, *args)
    for args, kind, match in [
            ((cache, start, cu, q[:, :3], q), ValueError, "q"), ((cache, start, cu, q, q3), ValueError, "o: shape"),
            ((cache, start, None, zeros(4, 4, 64), zeros(4, 4, 64)), ValueError, "need cu_tokens"),
            ((cache, start, cu, q, q.clone()), ValueError, "CUDA")]:
        with pytest.raises(kind, match=match):
            lq.lq_attn_prefill(cfg, *args)


def test_token_strides():
    from linear_attention_recurrent_int8_b200.attention import _rows
    cfg = lq.AttnConfig(4, 2, 64)
    qkv = zeros(3, 5, 8 * 64)
    assert _rows(qkv[..., :256].unflatten(-1, (4, 64)), "q", cfg, 4) == (15, 512)
    assert _rows(qkv[:1, :1, :256].unflatten(-1, (4, 64)), "q", cfg, 4) == (1, 256)
    assert _rows(qkv[:, :1, 256:384].unflatten(-1, (2, 64)), "k", cfg, 2) == (3, 2560)
    assert _rows(zeros(0, 4, 64), "q", cfg, 4) == (0, 256)


# ------------------------------------------------------------------ the reference itself

def test_reference_attention_by_hand():
    q = torch.tensor([[1.0, 0.0]], dtype=torch.float64)
    K = torch.tensor([[0.0, 5.0], [2.0, 0.0], [9.0, 9.0]], dtype=torch.float64)
    V = torch.tensor([[1.0, 0.0], [0.0, 1.0], [7.0, 7.0]], dtype=torch.float64)
    mask = torch.tensor([[True, True, False]])
    o, av, mag = ref.attend(q, K, V, mask, 0.5, 0.0)
    e = 2.718281828459045
    assert torch.allclose(o, torch.tensor([[1 / (1 + e), e / (1 + e)]], dtype=torch.float64))
    assert torch.equal(o, av) and mag.item() == 1.0


def test_reference_rotation_by_hand():
    x = torch.tensor([[[3.0, 4.0] + [0.0] * 14]], dtype=torch.float64)
    cs = torch.zeros(2, 16)
    cs[1, 8:] = 1.0  # a quarter turn at position 1
    y, _ = ref.norm_rotate(x, 1, 0.0, None, 16, True, cs, torch.tensor([1]))
    assert torch.allclose(y[0, 0, :2], torch.tensor([-0.8, 0.6], dtype=torch.float64))
    y, _ = ref.norm_rotate(x, 0, 0.0, None, 16, False, cs, torch.tensor([1]))
    assert y[0, 0, 8] == 3.0 and y[0, 0, 9] == 4.0 and y[0, 0, 0] == 0.0


@pytest.mark.parametrize("change", [dict(softcap=1e-4), dict(softcap=2e6), dict(softcap=float("inf")), dict(scale=-2e6),
                                    dict(scale=float("nan"))])
def test_scales_and_caps_out_of_range_are_refused(change):
    assert decode_call(cfg_c(**change), cache_c()) == INVALID
    assert prefill_call(cfg_c(**change), cache_c()) == INVALID


def test_the_smallest_eps():
    assert norm_call(cfg_c(norm=lq.LQ_NORM_L2, eps=1e-31)) == INVALID
    assert norm_call(cfg_c(norm=lq.LQ_NORM_L2, eps=1e-30), tokens=0) == OK


@pytest.mark.parametrize("change", [dict(window=1 << 32), dict(window=(1 << 32) + 5), dict(window=1 << 63), dict(q_heads=(1 << 32) + 8),
                                    dict(rot_dim=1 << 40), dict(norm=(1 << 32) + 1), dict(softcap=1e-60)])
def test_values_past_the_fields_of_the_struct_are_refused(change):
    """A window of 2^32 would be cut off to 0, which is none; so would a cap
    below the range of float."""
    with pytest.raises(ValueError, match=next(iter(change))):
        lq.AttnConfig(**{**dict(q_heads=8, kv_heads=2), **change})
    with pytest.raises(ValueError, match="batch"):
        lq.lq_attn_workspace_bytes(lq.AttnConfig(8, 2), (1 << 32) + 4)
    assert lq.AttnConfig(8, 2, window=(1 << 31) - 1).c().window == (1 << 31) - 1
    kp = torch.empty(1, 2, 16, 128, dtype=torch.bfloat16, device="meta")
    with pytest.raises(ValueError, match="max_pages"):
        lq.KvCache(lq.AttnConfig(8, 2), kp, kp, torch.empty(1, (1 << 32) + 4, dtype=torch.int32, device="meta"))


def test_calls_without_sequences_or_heads_are_refused():
    cfg = lq.AttnConfig(4, 2, 64)
    kp = zeros(9, 2, 16, 64)
    none = lq.KvCache(cfg, kp, kp.clone(), zeros(0, 5, dtype=torch.int32))
    q, k, pos = zeros(6, 4, 64), zeros(6, 2, 64), zeros(0, dtype=torch.int32)
    with pytest.raises(ValueError, match="0 sequences"):
        lq.lq_kv_append(cfg, none, pos, None, None, k, k, None, None, None, None)
    with pytest.raises(ValueError, match="0 sequences"):
        lq.lq_attn_prefill(cfg, none, pos, None, q, q)
    some = lq.KvCache(cfg, kp, kp.clone(), zeros(3, 5, dtype=torch.int32))
    with pytest.raises(ValueError, match="q: shape"):
        lq.lq_attn_prefill(lq.AttnConfig(0, 2, 64), some, zeros(3, dtype=torch.int32), None, q, q)
