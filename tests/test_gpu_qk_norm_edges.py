"""The query/key norm with rotation on the GPU at the edges of its range.
Checks and tolerances are those of test_gpu_qk_norm."""
from __future__ import annotations

import pytest
import torch

import structured_sparse_state_amd as pk
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


def test_more_rows_than_one_launch_has_threads_for():
    """2^30 rows and some, of one value each, in place."""
    L = (1 << 30) + 1000
    x = torch.randn((1, 1, L, 1), device="cuda:0", dtype=torch.bfloat16)
    none = torch.empty((1, 0, L, 1), device="cuda:0", dtype=torch.bfloat16)
    print("[case] 2^30 rows", flush=True)
    parts = [slice(0, 1 << 20), slice((1 << 29) - 1000, (1 << 29) + 1000), slice(L - (1 << 20), L)]
    want = [x[:, :, p].double() / (x[:, :, p].double() ** 2 + 0.25).sqrt() for p in parts]
    total = 0.0
    for n in range(0, L, 1 << 26):
        y = x[:, :, n:n + (1 << 26)].float()
        total += float((y / (y * y + 0.25).sqrt()).double().square().sum())
    pk.qk_norm_rope(x, none, eps=0.25, out=(x, none))
    torch.cuda.synchronize()
    for p, w in zip(parts, want):
        assert ((x[:, :, p].double() - w).abs() <= (2.0 ** -8 + 1e-5) * w.abs()).all()
    # every row once: a row taken twice is another value
    got = sum(float(x[:, :, n:n + (1 << 26)].double().square().sum()) for n in range(0, L, 1 << 26))
    assert abs(got - total) <= 2.0 ** -7 * total
