"""More calls that the cache in pages refuses, on the host (without a GPU)."""
import math

import pytest

from test_paged_refusals import _abi, fwd_args, refused


@pytest.mark.parametrize("cap", [2.0 ** 126, 1e38, 3.4e38, math.inf, math.nan, -1.0])
def test_caps_that_log2_units_do_not_hold(cap):
    abi = _abi()
    refused(abi, "bsa_paged_fwd", fwd_args(abi, logits_soft_cap=cap), "INVALID_ARG")
