"""Host-side checks of the norm, the key/value cache and the attention: arguments that are refused before any GPU
work (fake pointers, never dereferenced), and tensors that the binding refuses."""
import ctypes

import pytest
import torch

A = 0x10000  # aligned fake device address


@pytest.fixture(scope="module")
def lib():
    from int8_mixed_precision_rowwise_b200 import build as b
    b.build()
    import int8_mixed_precision_rowwise_b200 as m
    return m


def test_norm_argument_errors(lib):
    f = lib._add_rmsnorm_quantize
    ws = lib.quantize_workspace_size(32, 64)

    def call(X=A, R=A, W=A, kind=0, rows=32, cols=64, eps=1e-6, t=6.0, h=A, Y=A, codes=A, absmax=A, bitmap=A, wsp=A,
             wsb=ws):
        return f(X, R, W, kind, rows, cols, eps, t, h, Y, codes, absmax, bitmap, wsp, wsb, None)

    for bad in (dict(X=None), dict(W=None), dict(codes=None), dict(absmax=None), dict(wsp=None), dict(Y=None),
                dict(bitmap=None), dict(kind=2), dict(kind=-1), dict(rows=-1), dict(eps=-1.0), dict(eps=float("nan")),
                dict(eps=float("inf"))):
        assert call(**bad) == lib.ERR_INVALID_ARG, bad
    for bad in (dict(cols=60), dict(cols=0), dict(cols=133152), dict(rows=1 << 31)):
        assert call(**bad) == lib.ERR_UNSUPPORTED_SHAPE, bad
    for bad in (dict(X=A + 8), dict(R=A + 2), dict(W=A + 4), dict(h=A + 8), dict(Y=A + 8), dict(codes=A + 4),
                dict(absmax=A + 4), dict(bitmap=A + 4), dict(wsp=A + 4)):
        assert call(**bad) == lib.ERR_ALIGNMENT, bad
    assert call(wsb=ws - 256) == lib.ERR_WORKSPACE
    assert call(rows=0, t=0.0, bitmap=None) == lib.OK


def test_dequantize_argument_errors(lib):
    f = lib._dequantize_rowwise
    assert f(None, A, 4, 64, 0, A, None) == lib.ERR_INVALID_ARG
    assert f(A, A, 4, 64, 5, A, None) == lib.ERR_INVALID_ARG
    assert f(A, A, 4, 60, 0, A, None) == lib.ERR_UNSUPPORTED_SHAPE
    assert f(A, A, 4, 64, 0, A + 8, None) == lib.ERR_ALIGNMENT
    assert f(A, A, 0, 64, 0, A, None) == lib.OK


def cache(lib, **change):
    c = dict(k_codes=A, v_codes=A, k_absmax=A, v_absmax=A, pages=10, heads=2, page_size=16, head_dim=64, batch=3,
             table_width=4, table_stride=4, page_table=A, seq_lens=A, cu_rows=A)
    c.update(change)
    return lib._KvCache(**c)


BAD_CACHES = [
    ("ERR_INVALID_ARG", [dict(pages=-1), dict(batch=-1), dict(table_width=-1), dict(table_stride=3),
                         dict(k_codes=None), dict(v_codes=None), dict(k_absmax=None), dict(v_absmax=None),
                         dict(page_table=None), dict(seq_lens=None), dict(cu_rows=None)]),
    ("ERR_UNSUPPORTED_SHAPE", [dict(head_dim=96), dict(head_dim=256), dict(page_size=8), dict(page_size=48),
                               dict(page_size=256), dict(heads=0), dict(heads=65536), dict(pages=1 << 31),
                               dict(pages=1 << 26), dict(table_width=1 << 27, table_stride=1 << 27)]),
    ("ERR_ALIGNMENT", [dict(k_codes=A + 8), dict(v_codes=A + 4), dict(k_absmax=A + 2), dict(v_absmax=A + 1),
                       dict(page_table=A + 2), dict(seq_lens=A + 2), dict(cu_rows=A + 2)]),
]


def entry_points(lib):
    ref = ctypes.byref
    ws = lib.kv_attention_workspace_size(4, 2, 64)

    def append(c, tokens=5, K=A, V=A, kind=0, s=(128, 64, 128, 64), wsp=A, wsb=256):
        return lib._kv_append(ref(c), K, V, kind, tokens, *s, wsp, wsb, None)

    def read(c, tokens=5, K=A, V=A, kind=0, wsp=A, wsb=256):
        return lib._kv_read(ref(c), K, V, kind, tokens, wsp, wsb, None)

    def attend(c, tokens=5, Q=A, kind=0, heads=4, s=(256, 64), scale=0.1, slopes=None, max_new=0, out=A, lse=None,
               wsp=A, wsb=ws):
        return lib._kv_attention(ref(c), Q, kind, tokens, heads, *s, scale, 1, slopes, max_new, out, lse, wsp, wsb, None)

    return append, read, attend


@pytest.mark.parametrize("which", [0, 1, 2])
def test_cache_argument_errors(lib, which):
    f = entry_points(lib)[which]
    for status, changes in BAD_CACHES:
        for change in changes:
            assert f(cache(lib, **change)) == getattr(lib, status), change
    good = cache(lib)
    assert f(good, tokens=-1) == lib.ERR_INVALID_ARG
    assert f(good, tokens=1 << 31) == lib.ERR_UNSUPPORTED_SHAPE
    assert f(good, kind=2) == lib.ERR_INVALID_ARG
    assert f(good, wsp=None) == lib.ERR_INVALID_ARG
    assert f(good, wsp=A + 8) == lib.ERR_ALIGNMENT
    assert f(good, wsb=255) == lib.ERR_WORKSPACE
    assert f(good, tokens=0) == lib.OK
    assert f(cache(lib, batch=0)) == lib.OK


def test_row_argument_errors(lib):
    append, read, attend = entry_points(lib)
    good = cache(lib)
    assert append(good, K=None) == lib.ERR_INVALID_ARG and append(good, V=None) == lib.ERR_INVALID_ARG
    assert append(good, K=A + 8) == lib.ERR_ALIGNMENT
    for s in ((132, 64, 128, 64), (128, 60, 128, 64), (128, 64, -128, 64), (128, 64, 128, 4)):
        assert append(good, s=s) == lib.ERR_ALIGNMENT
    assert read(good, K=None) == lib.ERR_INVALID_ARG and read(good, V=A + 8) == lib.ERR_ALIGNMENT
    for bad in (dict(Q=None), dict(out=None), dict(heads=0), dict(heads=-2), dict(scale=float("nan")),
                dict(scale=float("inf")), dict(max_new=-1)):
        assert attend(good, **bad) == lib.ERR_INVALID_ARG, bad
    for bad in (dict(heads=3), dict(heads=65538), dict(heads=8, tokens=1 << 29)):
        assert attend(good, **bad) == lib.ERR_UNSUPPORTED_SHAPE, bad
    for bad in (dict(Q=A + 2), dict(out=A + 8), dict(s=(256, 4)), dict(s=(-256, 64)), dict(slopes=A + 2),
                dict(lse=A + 2)):
        assert attend(good, **bad) == lib.ERR_ALIGNMENT, bad
    assert attend(good, wsb=lib.kv_attention_workspace_size(4, 2, 64) - 1) == lib.ERR_WORKSPACE
    assert lib.kv_attention_workspace_size(0, 2, 64) == 0


def test_binding_refuses_cpu_tensors(lib):
    x = torch.zeros((4, 64), dtype=torch.float16)
    with pytest.raises(TypeError):
        lib.add_rmsnorm_quantize(x, x[0])
    with pytest.raises(TypeError):
        lib.dequantize_rowwise(torch.zeros((4, 64), dtype=torch.int8), torch.zeros(4))
    c = torch.zeros((2, 1, 16, 64), dtype=torch.int8)
    a, i = torch.zeros((2, 1)), torch.zeros((1, 2), dtype=torch.int32)
    q = torch.zeros((1, 1, 64), dtype=torch.float16)
    with pytest.raises(TypeError):
        lib.kv_append(q, q, c, c, a, a, i, i[0, :1], i[0])
    with pytest.raises(TypeError):
        lib.kv_read(c, c, a, a, i, i[0, :1], i[0], 1)
    with pytest.raises(TypeError):
        lib.kv_attention(q, c, c, a, a, i, i[0, :1], i[0])


def test_workspaces_that_do_not_fit_are_refused(lib):
    for bad in (torch.zeros(4096, dtype=torch.uint8), torch.zeros(4096, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError):
            lib._workspace(bad, 0)


def test_streams_outside_of_captures_have_no_number(lib):
    assert lib.load()["_stream_capture_id"](None) == 0
