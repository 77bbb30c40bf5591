"""The query/key norm with rotation on the GPU at the edges of its range.
Checks and tolerances are those of test_gpu_qk_norm."""
from __future__ import annotations

import pytest

from tests.test_gpu_qk_norm import TYPES, check, inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("pairs", ["half", "adjacent"])
@pytest.mark.parametrize("R", [2, 20, 24, 30, 32])
def test_later_rows_of_a_table(dtype, pairs, R):
    """cos[t:] of a table, where its rows are not whole 16-byte units too."""
    print(f"[case] R={R} {pairs} {dtype}", flush=True)
    c, dq, dk = inputs(R, 2, 3, 1, 9, 64, R, TYPES[dtype])
    for first in (1, 2, 3):
        x = {**c, "cos": c["cos"][first:], "sin": c["sin"][first:]}
        assert x["cos"].is_contiguous() and x["cos"].data_ptr() % 16 == first * R * 2 % 16
        check(x, dq, dk, "rms", pairs, dtype)
