"""Paged-cache calls that are refused before any launch, and the errors that name them (CPU only), beside those of
tests/test_paged_checks.py."""
import ctypes

import pytest

from test_paged_checks import ALIGN, c_pages, library  # noqa: F401 (the fixture builds the library)

_P = ctypes.c_void_p


@pytest.mark.parametrize("k,v", [(4104, 4096), (4096, 4104), (4098, 4112), (4120, 4120)])
def test_c_gather_outputs_are_16_byte_aligned(library, k, v):  # noqa: F811
    assert library.flashmask_paged_gather(ctypes.byref(c_pages()), _P(4096), 5, _P(k), _P(v), None) == ALIGN
