"""Paged key/value cache: append with rotation, attention, gather.

For serving a model trained with column-sparse masks.  The cache is a pair of
plain tensors, ``k_pages`` and ``v_pages``:

  bf16    ``[P, Hkv, page_size, d]`` bfloat16
  4 bits  ``[P, Hkv, page_size, d // 2]`` uint8 (byte i of a row: the codes of
          values 2i, low half, and 2i + 1) with ``k_scales``, ``v_scales``
          ``[P, Hkv, page_size, 2]`` bfloat16 (scale and minimum of each row; a
          code c stands for minimum + scale * c)

``block_table`` ``[B, M]`` int32 hands pages to sequences: position j of
sequence b is slot ``j % page_size`` of page ``block_table[b, j // page_size]``.
The calls run on the current stream of the tensors' device, allocate only
their outputs and workspace (or take them), never synchronise and can be
captured in a CUDA graph.  They record no gradient.  Table entries, positions
and lengths out of range are reported by ``get_status()`` (-9), with the
tokens concerned left out.
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple

import torch

from ._binding import _check, load_library

_BF16, _I32, _F32, _U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
_P, _LL, _I = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32


class _Pages(ctypes.Structure):
    _fields_ = [("k", _P), ("v", _P), ("k_scales", _P), ("v_scales", _P), ("table", _P), ("table_stride", _LL)] + \
        [(n, _I) for n in ("B", "table_width", "num_pages", "page_size", "Hkv", "d", "bits")]


class _Append(ctypes.Structure):
    _fields_ = [("q", _P), ("k", _P), ("v", _P), ("q_strides", _LL * 3), ("k_strides", _LL * 3),
                ("v_strides", _LL * 3), ("q_out", _P), ("start", _P), ("counts", _P), ("positions", _P), ("cos", _P),
                ("sin", _P), ("N", _I), ("Hq", _I), ("rot", _I), ("table_len", _I), ("interleaved", _I)]


class _Rows(ctypes.Structure):
    _fields_ = [("q", _P), ("q_strides", _LL * 3), ("lens", _P), ("start", _P), ("lts", _P), ("lte", _P),
                ("uts", _P), ("ute", _P), ("Nq", _I), ("Hq", _I), ("Hm", _I), ("Nm", _I), ("causal", _I),
                ("scale", ctypes.c_float), ("o", _P), ("lse", _P)]


def _is(name: str, t, dtype, shape) -> None:
    """Type, dtype and shape (None: any size) of one argument; the kernels trust these sizes."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    have = t.shape
    if len(have) != len(shape) or any(w is not None and w != h for w, h in zip(shape, have)):
        want = ", ".join("*" if w is None else str(w) for w in shape)
        raise ValueError(f"{name} must have shape [{want}], got {list(have)}")


def _placed(dev, named) -> None:
    """Every tensor on the CUDA device `dev` and contiguous."""
    for n, t in named:
        if t is None:
            continue
        if t.device != dev:
            raise ValueError(f"{n} is on {t.device}, expected {dev}")
        if not t.is_contiguous():
            raise ValueError(f"{n} must be contiguous")


def _strides(name: str, t: torch.Tensor):
    """{batch, token, head} strides of rows [B, N, H, d]; any, as long as 16-byte loads stay aligned."""
    s = t.stride()
    if s[3] != 1:
        raise ValueError(f"{name} must have unit stride over its last dimension")
    sh = t.shape
    r = (s[0] if sh[0] > 1 else 0, s[1] if sh[1] > 1 else 0, s[2] if sh[2] > 1 else 0)
    if (r[0] | r[1] | r[2]) & 7 or t.data_ptr() & 15:
        raise ValueError(f"{name}: strides must be multiples of 8 elements and the data 16-byte aligned")
    return r


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _pages(k_pages, v_pages, k_scales, v_scales, block_table, B=None, d=None, Hkv=None, Hq=None):
    """Checks the cache and its table, against the caller's sizes where given; returns the C structure
    and the sizes it holds."""
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("k_pages must be a 4-D tensor [P, Hkv, page_size, d]")
    P, H, page, last = k_pages.shape
    if k_pages.dtype is _U8:
        bits, width = 4, 2 * last
        _is("k_scales", k_scales, _BF16, (P, H, page, 2))
        _is("v_scales", v_scales, _BF16, (P, H, page, 2))
    else:
        bits, width = 16, last
        _is("k_pages", k_pages, _BF16, (P, H, page, last))
        if k_scales is not None or v_scales is not None:
            raise ValueError("k_scales and v_scales belong to 4-bit pages (uint8)")
    _is("v_pages", v_pages, k_pages.dtype, (P, H, page, last))
    if d is not None and d != width:
        raise ValueError(f"pages hold heads of {width} values, expected {d}")
    _is("block_table", block_table, _I32, (None, None))
    M = block_table.shape[1]
    if B is not None and B != block_table.shape[0]:
        raise ValueError(f"block_table is for {block_table.shape[0]} sequences, expected {B}")
    B = block_table.shape[0]
    if Hkv is not None and Hkv != H:
        raise ValueError(f"k has {Hkv} heads, the cache {H}")
    if Hq is not None and Hq % H:
        raise ValueError(f"q has {Hq} heads, which {H} heads of the cache do not divide")
    if M > 1 and block_table.stride(1) != 1:
        raise ValueError("block_table must have unit stride over its last dimension")
    if not k_pages.is_cuda:
        raise TypeError("k_pages must be a CUDA tensor")
    dev = k_pages.device
    _placed(dev, (("k_pages", k_pages), ("v_pages", v_pages), ("k_scales", k_scales), ("v_scales", v_scales)))
    if block_table.device != dev:
        raise ValueError(f"block_table is on {block_table.device}, expected {dev}")
    c = _Pages(k_pages.data_ptr(), v_pages.data_ptr(), _ptr(k_scales), _ptr(v_scales), block_table.data_ptr(),
               block_table.stride(0) if B > 1 else 0, B, M, P, page, H, width, bits)
    return c, B, H, width, dev


def _call(name: str, dev, *args) -> None:
    """Runs one entry point on the current stream of `dev`, with that device current."""
    fn = getattr(load_library(), name)
    if torch.cuda.current_device() == dev.index:
        rc = fn(*args, torch.cuda.current_stream(dev).cuda_stream)
    else:
        with torch.cuda.device(dev):
            rc = fn(*args, torch.cuda.current_stream(dev).cuda_stream)
    _check(rc, name)


def paged_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                 block_table: torch.Tensor, start: torch.Tensor, *, counts: Optional[torch.Tensor] = None,
                 q: Optional[torch.Tensor] = None, cos: Optional[torch.Tensor] = None,
                 sin: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                 interleaved: bool = False, k_scales: Optional[torch.Tensor] = None,
                 v_scales: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None):
    """Appends k, v ``[B, N, Hkv, d]`` (bf16, any strides) to the pages; token i of sequence b goes to
    position ``start[b] + i``.  ``counts`` ``[B]``: how many of the N tokens are real (the others are padding
    and touch no page).

    With ``cos``, ``sin`` ``[n, rot / 2]`` fp32 the first ``rot`` values of each row of k, and of
    ``q`` ``[B, N, Hq, d]`` if given, are rotated by the angles of the token's rotation position:
    ``positions`` ``[B, N]`` int32, or start + i.  Pairs are values (i, i + rot/2), or neighbours with
    ``interleaved``.  Returns the rotated q (padding rows 0; written to ``q_out`` if given, which may be a
    contiguous q itself), or None without q."""
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be a 4-D tensor [B, N, Hkv, d]")
    B, N, Hkv, d = k.shape
    _is("k", k, _BF16, (B, N, Hkv, d))
    _is("v", v, _BF16, (B, N, Hkv, d))
    _is("start", start, _I32, (B,))
    Hq = 0
    if q is not None:
        _is("q", q, _BF16, (B, N, None, d))
        Hq = q.shape[2]
        if q_out is not None:
            _is("q_out", q_out, _BF16, (B, N, Hq, d))
    elif q_out is not None:
        raise ValueError("q_out without q")
    if counts is not None:
        _is("counts", counts, _I32, (B,))
    rot = n_pos = 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin must be given together")
    if cos is not None:
        _is("cos", cos, _F32, (None, None))
        _is("sin", sin, _F32, cos.shape)
        n_pos, rot = cos.shape[0], 2 * cos.shape[1]
    if positions is not None:
        if cos is None:
            raise ValueError("positions without cos and sin")
        _is("positions", positions, _I32, (B, N))
    ks, vs = _strides("k", k), _strides("v", v)
    qs = (0, 0, 0) if q is None else _strides("q", q)
    pages, _, _, _, dev = _pages(k_pages, v_pages, k_scales, v_scales, block_table, B, d, Hkv)
    for n, t in (("k", k), ("v", v), ("q", q)):
        if t is not None and t.device != dev:
            raise ValueError(f"{n} is on {t.device}, expected {dev}")
    _placed(dev, (("start", start), ("counts", counts), ("cos", cos), ("sin", sin), ("positions", positions),
                  ("q_out", q_out)))
    if q is not None and q_out is None:
        q_out = torch.empty((B, N, Hq, d), dtype=_BF16, device=dev)
    c = _Append(_ptr(q), k.data_ptr(), v.data_ptr(), qs, ks, vs, _ptr(q_out), start.data_ptr(), _ptr(counts),
                _ptr(positions), _ptr(cos), _ptr(sin), N, Hq, rot, n_pos, 1 if interleaved else 0)
    _call("flashmask_paged_append", dev, ctypes.byref(pages), ctypes.byref(c))
    return q_out


def _rows(q, lens, start, lts, lte, uts, ute):
    B, Hq = q.shape[0], q.shape[2]
    _is("q", q, _BF16, (B, None, Hq, None))
    _is("lens", lens, _I32, (B,))
    if start is not None:
        _is("start", start, _I32, (B,))
    Hm, Nm = 1, 0
    vecs = (("lts", lts), ("lte", lte), ("uts", uts), ("ute", ute))
    ref = next((x for _, x in vecs if x is not None), None)
    if ref is not None:
        if not isinstance(ref, torch.Tensor) or ref.dim() != 3:
            raise ValueError("mask vectors must be 3-D tensors [B, Hm, Nm]")
        Hm, Nm = ref.shape[1], ref.shape[2]
        for n, x in vecs:
            if x is not None:
                _is(n, x, _I32, (B, Hm, Nm))
        if (lts is None) != (lte is None) or (uts is None) != (ute is None):
            raise ValueError("lts and lte, and uts and ute, must be given together")
        if Hm not in (1, Hq):
            raise ValueError(f"mask vectors have {Hm} heads, expected 1 or {Hq}")
    return Hm, Nm, vecs


def paged_attention(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor,
                    lens: torch.Tensor, lts=None, lte=None, uts=None, ute=None, scale: Optional[float] = None, *,
                    start: Optional[torch.Tensor] = None, causal: bool = True,
                    k_scales: Optional[torch.Tensor] = None, v_scales: Optional[torch.Tensor] = None,
                    out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None,
                    workspace: Optional[torch.Tensor] = None):
    """Rows q ``[B, Nq, Hq, d]`` (bf16, any strides; one per sequence, or a short run) over the first
    ``lens[b]`` cached keys -> (o ``[B, Nq, Hq, d]`` bf16, lse ``[B, Hq, Nq]`` fp32).

    Row i of sequence b stands at position p = ``start[b] + i`` (default: the last Nq of the ``lens[b]``
    tokens) and sees key j iff j <= p (unless ``causal`` is False) and neither LTS[j] <= p < LTE[j] nor
    UTS[j] <= p < UTE[j], with mask vectors ``[B, Hm, Nm]`` as in ``fwd`` (keys from Nm on: no
    interval).  A row that sees nothing gives 0 and -inf; what unseen keys hold has no influence."""
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a 4-D tensor [B, Nq, Hq, d]")
    B, Nq, Hq, d = q.shape
    Hm, Nm, vecs = _rows(q, lens, start, lts, lte, uts, ute)
    qs = _strides("q", q)
    if out is not None:
        o, lse = out
        _is("o", o, _BF16, (B, Nq, Hq, d))
        _is("lse", lse, _F32, (B, Hq, Nq))
    pages, _, _, _, dev = _pages(k_pages, v_pages, k_scales, v_scales, block_table, B, d, Hq=Hq)
    if q.device != dev:
        raise ValueError(f"q is on {q.device}, expected {dev}")
    if out is None:
        o = torch.empty((B, Nq, Hq, d), dtype=_BF16, device=dev)
        lse = torch.empty((B, Hq, Nq), dtype=_F32, device=dev)
    _placed(dev, (("lens", lens), ("start", start), *vecs, ("o", o), ("lse", lse), ("workspace", workspace)))
    c = _Rows(q.data_ptr(), qs, lens.data_ptr(), _ptr(start), _ptr(lts), _ptr(lte), _ptr(uts),
              _ptr(ute), Nq, Hq, Hm, Nm, 1 if causal else 0, scale or 0.0, o.data_ptr(), lse.data_ptr())
    pp, cp = ctypes.byref(pages), ctypes.byref(c)
    if workspace is None:
        need = load_library().flashmask_paged_attention_workspace_size(pp, cp)
        workspace = torch.empty(max(need, 256), dtype=_U8, device=dev)
    _call("flashmask_paged_attention", dev, pp, cp, workspace.data_ptr(), workspace.numel() * workspace.element_size())
    return o, lse


def paged_gather(k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor,
                 N: int, *, k_scales: Optional[torch.Tensor] = None, v_scales: Optional[torch.Tensor] = None,
                 out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """The first N positions of each sequence as dense (k, v) ``[B, N, Hkv, d]`` bf16, as ``fwd`` and ``bwd``
    take them: positions from ``lens[b]`` on are 0; 4-bit pages give the values their codes stand for."""
    _is("lens", lens, _I32, (None,))
    pages, B, Hkv, d, dev = _pages(k_pages, v_pages, k_scales, v_scales, block_table)
    _is("lens", lens, _I32, (B,))
    if N < 0:
        raise ValueError("N must not be negative")
    if out is not None:
        k, v = out
        _is("k", k, _BF16, (B, N, Hkv, d))
        _is("v", v, _BF16, (B, N, Hkv, d))
    else:
        k = torch.empty((B, N, Hkv, d), dtype=_BF16, device=dev)
        v = torch.empty((B, N, Hkv, d), dtype=_BF16, device=dev)
    _placed(dev, (("lens", lens), ("k", k), ("v", v)))
    _call("flashmask_paged_gather", dev, ctypes.byref(pages), lens.data_ptr(), N, k.data_ptr(), v.data_ptr())
    return k, v
