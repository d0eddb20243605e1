"""The paged-cache entry points reject malformed arguments before any launch (CPU only): the
Python binding by exceptions, the C ABI by error codes."""
import ctypes
import sys

import pytest
import torch

import column_sparse_masked_b200 as fm

_P, _LL, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class _Pages(ctypes.Structure):  # flashmask_pages
    _fields_ = [("k", _P), ("v", _P), ("k_scales", _P), ("v_scales", _P), ("table", _P), ("table_stride", _LL)] + \
        [(n, _I) for n in ("B", "table_width", "num_pages", "page_size", "Hkv", "d", "bits")]


class _Append(ctypes.Structure):  # flashmask_append
    _fields_ = [("q", _P), ("k", _P), ("v", _P), ("q_strides", _LL * 3), ("k_strides", _LL * 3),
                ("v_strides", _LL * 3), ("q_out", _P), ("start", _P), ("counts", _P), ("positions", _P), ("cos", _P),
                ("sin", _P), ("N", _I), ("Hq", _I), ("rot", _I), ("table_len", _I), ("interleaved", _I)]


class _Rows(ctypes.Structure):  # flashmask_paged_rows
    _fields_ = [("q", _P), ("q_strides", _LL * 3), ("lens", _P), ("start", _P), ("lts", _P), ("lte", _P),
                ("uts", _P), ("ute", _P), ("Nq", _I), ("Hq", _I), ("Hm", _I), ("Nm", _I), ("causal", _I),
                ("scale", ctypes.c_float), ("o", _P), ("lse", _P)]


B, N, HQ, HKV, D, P, PAGE, M = 2, 3, 4, 2, 64, 5, 16, 4
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def library():
    from column_sparse_masked_b200 import build

    build.build()
    return fm.load_library()


def args(bits=16):
    a = dict(k=torch.zeros(B, N, HKV, D, dtype=BF), v=torch.zeros(B, N, HKV, D, dtype=BF),
             q=torch.zeros(B, N, HQ, D, dtype=BF), block_table=torch.zeros(B, M, dtype=torch.int32),
             start=torch.zeros(B, dtype=torch.int32), lens=torch.zeros(B, dtype=torch.int32),
             cos=torch.zeros(99, D // 2), sin=torch.zeros(99, D // 2), k_scales=None, v_scales=None)
    shape, dt = ((P, HKV, PAGE, D), BF) if bits == 16 else ((P, HKV, PAGE, D // 2), torch.uint8)
    a["k_pages"], a["v_pages"] = torch.zeros(shape, dtype=dt), torch.zeros(shape, dtype=dt)
    if bits == 4:
        a["k_scales"], a["v_scales"] = (torch.zeros(P, HKV, PAGE, 2, dtype=BF) for _ in range(2))
    return a


def append(a, **kw):
    return fm.paged_append(a["k"], a["v"], a["k_pages"], a["v_pages"], a["block_table"], a["start"], q=a["q"],
                           cos=a["cos"], sin=a["sin"], k_scales=a["k_scales"], v_scales=a["v_scales"], **kw)


def attend(a, *masks, **kw):
    return fm.paged_attention(a["q"], a["k_pages"], a["v_pages"], a["block_table"], a["lens"], *masks,
                              k_scales=a["k_scales"], v_scales=a["v_scales"], **kw)


def gather(a, n=7, **kw):
    return fm.paged_gather(a["k_pages"], a["v_pages"], a["block_table"], a["lens"], n, k_scales=a["k_scales"],
                           v_scales=a["v_scales"], **kw)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("call", [append, attend, gather])
def test_well_formed_cpu_arguments_only_fail_on_the_device(call, bits):
    with pytest.raises(TypeError, match="CUDA"):
        call(args(bits))


BAD = [
    ("k_pages", lambda t: t.float(), "k_pages"), ("k_pages", lambda t: t[0], "k_pages"),
    ("v_pages", lambda t: t[:-1], "v_pages"), ("v_pages", lambda t: t.float(), "v_pages"),
    ("block_table", lambda t: t.long(), "block_table"), ("block_table", lambda t: t[0], "block_table"),
    ("k_scales", lambda t: torch.zeros(P, HKV, PAGE, 2, dtype=BF), "4-bit"),
]


@pytest.mark.parametrize("call", [append, attend, gather])
@pytest.mark.parametrize("name,change,match", BAD)
def test_bad_cache(call, name, change, match):
    a = args()
    a[name] = change(a[name])
    with pytest.raises((TypeError, ValueError), match=match):
        call(a)


@pytest.mark.parametrize("call", [append, attend, gather])
@pytest.mark.parametrize("name", ["k_scales", "v_scales"])
@pytest.mark.parametrize("change", [lambda t: None, lambda t: t.float(), lambda t: t[..., :1]])
def test_bad_scales(call, name, change):
    a = args(4)
    a[name] = change(a[name])
    with pytest.raises((TypeError, ValueError), match=name):
        call(a)


@pytest.mark.parametrize("name,change,match", [
    ("k", lambda t: t[:, :, :1], "v must"), ("k", lambda t: t.float(), "k must"), ("v", lambda t: t[:, :2], "v must"),
    ("q", lambda t: t[:1], "q must"), ("q", lambda t: t.half(), "q must"), ("start", lambda t: t.long(), "start"),
    ("start", lambda t: t[:1], "start"), ("cos", lambda t: None, "together"), ("sin", lambda t: t[:, :8], "sin"),
    ("cos", lambda t: t.double(), "cos"), ("block_table", lambda t: t[:1], "block_table is for"),
    ("k", lambda t: torch.zeros(B, N, HKV, D + 4, dtype=BF)[..., 1:D + 1], "k: strides"),
    ("q", lambda t: torch.zeros(B, N, HQ, D, 2, dtype=BF)[..., 0], "unit stride"),
])
def test_bad_append(name, change, match):
    a = args()
    a[name] = change(a[name])
    with pytest.raises((TypeError, ValueError), match=match):
        append(a)


def test_bad_append_options():
    a = args()
    for kw in (dict(counts=torch.zeros(B + 1, dtype=torch.int32)), dict(positions=torch.zeros(B, N + 1, dtype=torch.int32)),
               dict(positions=torch.zeros(B, N)), dict(q_out=torch.zeros(B, N, HQ, D)),
               dict(counts=torch.zeros(B, dtype=torch.int64))):
        with pytest.raises((TypeError, ValueError), match=next(iter(kw))):
            append(a, **kw)
    with pytest.raises(ValueError, match="k has 1 heads"):
        fm.paged_append(a["k"][:, :, :1], a["v"][:, :, :1], a["k_pages"], a["v_pages"], a["block_table"], a["start"])
    with pytest.raises(ValueError, match="q_out"):
        fm.paged_append(a["k"], a["v"], a["k_pages"], a["v_pages"], a["block_table"], a["start"], q_out=a["q"])
    with pytest.raises(ValueError, match="positions"):
        fm.paged_append(a["k"], a["v"], a["k_pages"], a["v_pages"], a["block_table"], a["start"],
                        positions=torch.zeros(B, N, dtype=torch.int32))


@pytest.mark.parametrize("name,change,match", [
    ("q", lambda t: t[0], "q must"), ("q", lambda t: t[:, :, :3], "q has"), ("q", lambda t: t[:1], "lens"),
    ("q", lambda t: torch.zeros(B, N, HQ, 128, dtype=BF), "pages hold"), ("lens", lambda t: t.long(), "lens"),
])
def test_bad_attention(name, change, match):
    a = args()
    a[name] = change(a[name])
    with pytest.raises((TypeError, ValueError), match=match):
        attend(a)


def test_bad_attention_masks_and_outputs():
    a = args()
    m = torch.zeros(B, 1, 30, dtype=torch.int32)
    for masks, match in (((m, None), "together"), ((m.long(), m.long()), "lts"), ((m, m[:, :, :5]), "lte"),
                         ((m[0], m[0]), "3-D"), ((None, None, m, None), "together"),
                         ((m.expand(B, 3, 30), m.expand(B, 3, 30)), "heads")):
        with pytest.raises((TypeError, ValueError), match=match):
            attend(a, *masks)
    with pytest.raises(ValueError, match="lse"):
        attend(a, out=(torch.zeros(B, N, HQ, D, dtype=BF), torch.zeros(B, N, HQ)))
    with pytest.raises(ValueError, match="start"):
        attend(a, start=torch.zeros(B + 1, dtype=torch.int32))


def test_bad_gather():
    a = args()
    with pytest.raises((TypeError, ValueError)):
        gather(a, n=-1)
    a["lens"] = a["lens"].long()
    with pytest.raises(TypeError, match="lens"):
        gather(a)


# ---- C ABI: codes, nothing launched ----
def c_pages(**kw):
    v = dict(k=4096, v=4096, k_scales=None, v_scales=None, table=4096, table_stride=M, B=B, table_width=M, num_pages=P,
             page_size=PAGE, Hkv=HKV, d=D, bits=16)
    v.update(kw)
    return _Pages(**v)


def c_append(**kw):
    s = (ctypes.c_int64 * 3)(N * HKV * D, HKV * D, D)
    v = dict(q=None, k=4096, v=4096, k_strides=s, v_strides=s, start=4096, cos=4096, sin=4096, N=N, Hq=HQ, rot=D,
             table_len=9, interleaved=0)
    v.update(kw)
    return _Append(**v)


def c_rows(**kw):
    s = (ctypes.c_int64 * 3)(N * HQ * D, HQ * D, D)
    v = dict(q=4096, q_strides=s, lens=4096, Nq=N, Hq=HQ, Hm=1, Nm=0, causal=1, scale=0.0, o=4096, lse=4096)
    v.update(kw)
    return _Rows(**v)


INVALID, UNSUPPORTED, ALIGN, WORKSPACE = -1, -2, -3, -4


@pytest.mark.parametrize("kw,code", [
    (dict(d=96), UNSUPPORTED), (dict(bits=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=8), UNSUPPORTED), (dict(page_size=512), UNSUPPORTED), (dict(B=-1), INVALID),
    (dict(Hkv=0), INVALID), (dict(num_pages=-1), INVALID), (dict(k=None), INVALID), (dict(table=None), INVALID),
    (dict(bits=4), INVALID), (dict(k=4104), ALIGN), (dict(table_width=1 << 27), UNSUPPORTED),
    (dict(num_pages=1 << 27), UNSUPPORTED), (dict(bits=4, k_scales=4104, v_scales=4096), ALIGN),
])
def test_c_pages(library, kw, code):
    pg = c_pages(**kw)
    p = ctypes.byref(pg)
    assert library.flashmask_paged_append(p, ctypes.byref(c_append()), None) == code
    assert library.flashmask_paged_gather(p, ctypes.c_void_p(4096), 5, ctypes.c_void_p(4096), ctypes.c_void_p(4096),
                                          None) == code
    assert library.flashmask_paged_attention_workspace_size(p, ctypes.byref(c_rows())) == 0
    assert library.flashmask_paged_attention(p, ctypes.byref(c_rows()), ctypes.c_void_p(4096), 1 << 30, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(start=None), INVALID), (dict(N=-1), INVALID),
    (dict(rot=24), UNSUPPORTED), (dict(rot=128), UNSUPPORTED), (dict(cos=None), INVALID), (dict(k=4098), ALIGN),
    (dict(k_strides=(ctypes.c_int64 * 3)(4, 8, 8)), ALIGN), (dict(v_strides=(ctypes.c_int64 * 3)(8, -8, 8)), INVALID),
    (dict(q=4096), INVALID), (dict(q=4096, q_out=4100), ALIGN), (dict(q=4096, q_out=4096, Hq=0), INVALID),
    (dict(interleaved=2), INVALID), (dict(N=1 << 30), UNSUPPORTED),
])
def test_c_append(library, kw, code):
    t = c_append(**kw)
    assert library.flashmask_paged_append(ctypes.byref(c_pages()), ctypes.byref(t), None) == code
    assert library.flashmask_paged_append(ctypes.byref(c_pages()), None, None) == INVALID
    assert library.flashmask_paged_append(None, ctypes.byref(t), None) == INVALID


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INVALID), (dict(lens=None), INVALID), (dict(o=None), INVALID), (dict(lse=None), INVALID),
    (dict(Hq=3), INVALID), (dict(Nq=-1), INVALID), (dict(causal=2), INVALID), (dict(q=4104), ALIGN),
    (dict(o=4104), ALIGN), (dict(lts=4096), INVALID), (dict(lts=4096, lte=4100), ALIGN),
    (dict(uts=4096, ute=4096, Hm=3, Nm=7), INVALID), (dict(Nq=1 << 30), UNSUPPORTED),
])
def test_c_attention(library, kw, code):
    r = c_rows(**kw)
    assert library.flashmask_paged_attention(ctypes.byref(c_pages()), ctypes.byref(r), ctypes.c_void_p(4096), 1 << 30,
                                             None) == code


def test_c_attention_workspace(library):
    pg, r = c_pages(), c_rows()
    need = library.flashmask_paged_attention_workspace_size(ctypes.byref(pg), ctypes.byref(r))
    assert need > 0
    call = library.flashmask_paged_attention
    assert call(ctypes.byref(pg), ctypes.byref(r), None, need, None) == WORKSPACE
    assert call(ctypes.byref(pg), ctypes.byref(r), ctypes.c_void_p(4096), need - 1, None) == WORKSPACE
    assert call(ctypes.byref(pg), ctypes.byref(r), ctypes.c_void_p(4096 + 16), need, None) == ALIGN


def test_c_empty_calls_touch_no_device(library):
    pg = c_pages(B=0)
    assert library.flashmask_paged_append(ctypes.byref(pg), ctypes.byref(c_append()), None) == 0
    assert library.flashmask_paged_append(ctypes.byref(c_pages()), ctypes.byref(c_append(N=0)), None) == 0
    assert library.flashmask_paged_gather(ctypes.byref(c_pages()), None, 0, None, None, None) == 0
    assert library.flashmask_paged_attention(ctypes.byref(c_pages()), ctypes.byref(c_rows(Nq=0)), None, 0, None) == 0


def test_missing_binding_is_named(monkeypatch):
    from column_sparse_masked_b200 import paged

    monkeypatch.setattr(paged, "_calls", None)
    monkeypatch.setitem(sys.modules, "column_sparse_masked_b200._paged_binding", None)
    monkeypatch.delattr(fm, "_paged_binding", raising=False)
    with pytest.raises(RuntimeError, match="_paged_binding.so is missing"):
        fm.paged_gather(None, None, None, None, 1)


@pytest.mark.parametrize("bits", [16, 4])
def test_pages_without_heads_are_refused(bits):
    a = args(bits)
    for n in ("k_pages", "v_pages", "k_scales", "v_scales"):
        if a[n] is not None:
            a[n] = a[n][:, :0]
    for call in (append, attend):
        with pytest.raises(ValueError, match="at least one head"):
            call(a)
