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
captured in a CUDA graph.  They record no gradient.  Tensors are contiguous and
16-byte aligned (a workspace: 256 bytes) where nothing else is said.  Table entries, positions
and lengths out of range are reported by ``get_status()`` (-9), with the
tokens concerned left out.
"""
from __future__ import annotations

import importlib
from typing import Optional, Tuple

import torch

from ._binding import FlashMaskError, load_library

_BF16, _I32, _F32, _U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8
_calls = None


def _load():
    """The compiled marshalling of these calls (_paged_binding.so), bound to the library in use."""
    global _calls
    lib = load_library()
    how = "build it with `python column_sparse_masked_b200/build.py"
    try:
        _paged_binding = importlib.import_module("._paged_binding", __package__)
    except ModuleNotFoundError as e:
        raise RuntimeError(f"_paged_binding.so is missing: {how}`") from e
    except ImportError as e:
        raise RuntimeError(f"_paged_binding.so does not load: {e}; {how} --force`") from e
    _paged_binding.bind(lib._name)
    _calls = _paged_binding
    return _calls


def _fail(code, where: str, explain, *args):
    """Raises for a call that did not run: the C ABI's error, or what is wrong with its arguments."""
    if code is not NotImplemented:
        raise FlashMaskError(code, where)
    explain(*args)
    raise ValueError(f"{where}: arguments are not of the documented kind")


# What the compiled marshalling checks, one by one, to name what it refused: types, dtypes and shapes whatever the
# device, then the device.
def _is(name: str, t, dtype, shape) -> None:
    """Type, dtype and shape (None: any size) of one argument."""
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


def _strides(name: str, t: torch.Tensor) -> None:
    """Rows [B, N, heads, d]: any strides, as long as 16-byte loads stay aligned."""
    if t.stride(3) != 1:
        raise ValueError(f"{name} must have unit stride over its last dimension")
    if any(t.shape[i] > 1 and t.stride(i) % 8 for i in range(3)) or t.data_ptr() % 16:
        raise ValueError(f"{name}: strides must be multiples of 8 elements and the data 16-byte aligned")


def _pages(k_pages, v_pages, k_scales, v_scales, block_table, B=None, d=None, Hkv=None, Hq=None):
    """The cache and its table, against the caller's sizes where given; returns its sizes and device."""
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise ValueError("k_pages must be a 4-D tensor [P, Hkv, page_size, d]")
    P, H, page, last = k_pages.shape
    if H == 0:
        raise ValueError("k_pages must have at least one head")
    if k_pages.dtype is _U8:
        width = 2 * last
        _is("k_scales", k_scales, _BF16, (P, H, page, 2))
        _is("v_scales", v_scales, _BF16, (P, H, page, 2))
    else:
        width = last
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
    return B, H, width, dev


def _explain_append(k, v, k_pages, v_pages, block_table, start, counts, q, cos, sin, positions, k_scales, v_scales, q_out):
    if not isinstance(k, torch.Tensor) or k.dim() != 4:
        raise ValueError("k must be a 4-D tensor [B, N, Hkv, d]")
    B, N, Hkv, d = k.shape
    _is("k", k, _BF16, (B, N, Hkv, d))
    _is("v", v, _BF16, (B, N, Hkv, d))
    _is("start", start, _I32, (B,))
    if q is not None:
        _is("q", q, _BF16, (B, N, None, d))
        if q_out is not None:
            _is("q_out", q_out, _BF16, (B, N, q.shape[2], d))
    elif q_out is not None:
        raise ValueError("q_out without q")
    if counts is not None:
        _is("counts", counts, _I32, (B,))
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin must be given together")
    if cos is not None:
        _is("cos", cos, _F32, (None, None))
        _is("sin", sin, _F32, cos.shape)
    if positions is not None:
        if cos is None:
            raise ValueError("positions without cos and sin")
        _is("positions", positions, _I32, (B, N))
    for n, t in (("k", k), ("v", v), ("q", q)):
        if t is not None:
            _strides(n, t)
    _, _, _, dev = _pages(k_pages, v_pages, k_scales, v_scales, block_table, B, d, Hkv)
    for n, t in (("k", k), ("v", v), ("q", q)):
        if t is not None and t.device != dev:
            raise ValueError(f"{n} is on {t.device}, expected {dev}")
    _placed(dev, (("start", start), ("counts", counts), ("cos", cos), ("sin", sin), ("positions", positions),
                  ("q_out", q_out)))


def _explain_attention(q, k_pages, v_pages, block_table, lens, lts, lte, uts, ute, start, k_scales, v_scales, o, lse,
                       workspace):
    if not isinstance(q, torch.Tensor) or q.dim() != 4:
        raise ValueError("q must be a 4-D tensor [B, Nq, Hq, d]")
    B, Nq, Hq, d = q.shape
    _is("q", q, _BF16, (B, Nq, Hq, d))
    _is("lens", lens, _I32, (B,))
    if start is not None:
        _is("start", start, _I32, (B,))
    vecs = (("lts", lts), ("lte", lte), ("uts", uts), ("ute", ute))
    ref = next((x for _, x in vecs if x is not None), None)
    if ref is not None:
        if not isinstance(ref, torch.Tensor) or ref.dim() != 3:
            raise ValueError("mask vectors must be 3-D tensors [B, Hm, Nm]")
        for n, x in vecs:
            if x is not None:
                _is(n, x, _I32, (B, ref.shape[1], ref.shape[2]))
        if (lts is None) != (lte is None) or (uts is None) != (ute is None):
            raise ValueError("lts and lte, and uts and ute, must be given together")
        if ref.shape[1] not in (1, Hq):
            raise ValueError(f"mask vectors have {ref.shape[1]} heads, expected 1 or {Hq}")
    _strides("q", q)
    if workspace is not None and not isinstance(workspace, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if o is not None or lse is not None:
        _is("o", o, _BF16, (B, Nq, Hq, d))
        _is("lse", lse, _F32, (B, Hq, Nq))
    _, _, _, dev = _pages(k_pages, v_pages, k_scales, v_scales, block_table, B, d, Hq=Hq)
    if q.device != dev:
        raise ValueError(f"q is on {q.device}, expected {dev}")
    _placed(dev, (("lens", lens), ("start", start), *vecs, ("o", o), ("lse", lse), ("workspace", workspace)))


def _explain_gather(k_pages, v_pages, block_table, lens, N, k_scales, v_scales, k, v):
    _is("lens", lens, _I32, (None,))
    if not isinstance(N, int):
        raise TypeError("N must be an integer")
    if N < 0:
        raise ValueError("N must not be negative")
    if N >= 1 << 31:
        raise ValueError("N must fit 32 bits")
    B, Hkv, d, dev = _pages(k_pages, v_pages, k_scales, v_scales, block_table)
    _is("lens", lens, _I32, (B,))
    if k is not None or v is not None:
        _is("k", k, _BF16, (B, N, Hkv, d))
        _is("v", v, _BF16, (B, N, Hkv, d))
    _placed(dev, (("lens", lens), ("k", k), ("v", v)))


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
    r = (_calls or _load()).append(k, v, k_pages, v_pages, block_table, start, counts, q, cos, sin, positions, interleaved,
                                   k_scales, v_scales, q_out)
    if r is None or isinstance(r, torch.Tensor):
        return r
    _fail(r, "flashmask_paged_append", _explain_append, k, v, k_pages, v_pages, block_table, start, counts, q, cos, sin,
          positions, k_scales, v_scales, q_out)


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
    o, lse = out or (None, None)
    r = (_calls or _load()).attention(q, k_pages, v_pages, block_table, lens, lts, lte, uts, ute, scale, start, causal,
                                      k_scales, v_scales, o, lse, workspace)
    if r.__class__ is tuple:
        return r
    _fail(r, "flashmask_paged_attention", _explain_attention, q, k_pages, v_pages, block_table, lens, lts, lte, uts, ute,
          start, k_scales, v_scales, o, lse, workspace)


def paged_gather(k_pages: torch.Tensor, v_pages: torch.Tensor, block_table: torch.Tensor, lens: torch.Tensor,
                 N: int, *, k_scales: Optional[torch.Tensor] = None, v_scales: Optional[torch.Tensor] = None,
                 out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None):
    """The first N positions of each sequence as dense (k, v) ``[B, N, Hkv, d]`` bf16, as ``fwd`` and ``bwd``
    take them: positions from ``lens[b]`` on are 0; 4-bit pages give the values their codes stand for."""
    k, v = out or (None, None)
    r = (_calls or _load()).gather(k_pages, v_pages, block_table, lens, N, k_scales, v_scales, k, v)
    if r.__class__ is tuple:
        return r
    _fail(r, "flashmask_paged_gather", _explain_gather, k_pages, v_pages, block_table, lens, N, k_scales, v_scales, k, v)
