"""Paged-cache calls that are refused before any launch, and the errors that name them (CPU only), beside those of
tests/test_paged_checks.py."""
import ctypes
import sys

import pytest
import torch

import column_sparse_masked_b200 as fm

from test_paged_checks import (ALIGN, UNSUPPORTED, args, attend, c_append, c_pages, c_rows, gather,  # noqa: F401
                               library)  # (the fixture builds the library)

_P = ctypes.c_void_p


@pytest.mark.parametrize("k,v", [(4104, 4096), (4096, 4104), (4098, 4112), (4120, 4120)])
def test_c_gather_outputs_are_16_byte_aligned(library, k, v):  # noqa: F811
    assert library.flashmask_paged_gather(ctypes.byref(c_pages()), _P(4096), 5, _P(k), _P(v), None) == ALIGN


def test_c_size_products_do_not_wrap(library):  # noqa: F811
    """Sizes whose product passes 64 bits are refused like those that pass 32: 2^30 x 2^30 tokens of 16 rows."""
    pg = c_pages(B=1 << 30, Hkv=4, num_pages=1)
    assert library.flashmask_paged_append(ctypes.byref(pg), ctypes.byref(c_append(N=1 << 30, q=4096, q_out=4096, Hq=8)),
                                          None) == UNSUPPORTED
    r = c_rows(Nq=1 << 30, Hq=16)
    assert library.flashmask_paged_attention_workspace_size(ctypes.byref(pg), ctypes.byref(r)) == 0
    assert library.flashmask_paged_attention(ctypes.byref(pg), ctypes.byref(r), _P(4096), 1 << 30, None) == UNSUPPORTED


def test_append_returns_a_q_out_of_any_tensor_class(monkeypatch):
    """q_out comes back also where it is a Parameter (the call had run, and an error was raised for it)."""
    from column_sparse_masked_b200 import paged

    class Calls:
        @staticmethod
        def append(*a):
            return a[-1]

    monkeypatch.setattr(paged, "_calls", Calls)
    out = torch.nn.Parameter(torch.zeros(2), requires_grad=False)
    assert paged.paged_append(*[None] * 6, q_out=out) is out


@pytest.mark.parametrize("workspace", [4096, "x", [torch.zeros(9)]])
def test_a_workspace_that_is_no_tensor_is_named(workspace):
    with pytest.raises(TypeError, match="workspace must be a torch.Tensor"):
        attend(args(), workspace=workspace)


@pytest.mark.parametrize("n", [2 ** 31, 2 ** 40])
def test_gather_of_more_positions_than_32_bits_is_named(n):
    with pytest.raises(ValueError, match="N must"):
        gather(args(), n=n)


def test_paged_calls_run_in_the_library_that_is_loaded(monkeypatch):
    """FLASHMASK_LIBRARY is read once: calls bound after a change of it still go to the library whose status
    get_status() reads."""
    from column_sparse_masked_b200 import paged

    bound = []

    class Binding:
        @staticmethod
        def bind(path):
            bound.append(path)

    loaded = fm.load_library()
    monkeypatch.setenv("FLASHMASK_LIBRARY", "checks" if "checks" not in loaded._name else "")
    monkeypatch.setattr(paged, "_calls", None)
    monkeypatch.setitem(sys.modules, "column_sparse_masked_b200._paged_binding", Binding)
    monkeypatch.setattr(fm, "_paged_binding", Binding, raising=False)
    paged._load()
    assert bound == [loaded._name]
