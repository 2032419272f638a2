"""Limits of the key/value cache calls, without a GPU."""
import pytest

import gemm_affine_int4_gb300 as g4
from test_kv_cpu import attention


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_block_tables_of_nearly_two_to_the_31_tokens(page):
    """Token numbers of a request, and the steps past its last tile, stay in 32 bits: wider tables are refused (without
    a workspace, so that the widest that is not refused ends there)."""
    widest = (2**31 - 4096) // page
    for width in (widest + 1, 2**31 // page - 1, 2**31 // page, 2**40):
        assert attention(page=page, width=width, ws=None) == g4.GAI4_ERR_INVALID_ARG
    assert attention(page=page, width=widest, ws=None) == g4.GAI4_ERR_WORKSPACE
