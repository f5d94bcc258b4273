"""The scan at channel counts whose last block is taken from a channel that no vector is aligned to, in
every number of states' form, against the 64-bit form (to the bounds of test_scan.py)."""
from __future__ import annotations

import pytest

from .test_scan import check

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("S,H,N,G,dtype,parts", [
    (37, 63, 5, 1, "bf16", {}),                   # eight channels a thread
    (20, 73, 8, 1, "fp16", {"gate": False}),
    (37, 69, 16, 1, "bf16", {}),                  # four
    (18, 202, 12, 2, "fp16", {}),
    (37, 95, 20, 1, "bf16", {}),                  # two
    (33, 67, 32, 1, "fp16", {"gate": False}),
    (600, 63, 16, 1, "bf16", {}),                 # in chunks
    (600, 61, 8, 1, "fp16", {}),
])
def test_odd_channel_counts(S, H, N, G, dtype, parts):
    check(S, 2, H, N, G, dtype, [S, S // 2], seed=S + H, **parts)
