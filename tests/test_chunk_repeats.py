"""The attention of chunks gives the same bits each time: some thousand calls of few items,
whose plans and parts are made anew each time."""
from __future__ import annotations

import pytest
import torch

import w4a16_weight_only_gemm_gb300 as w4
from test_chunk_attention import make

CALLS = 3000


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [[(700, 5)], [(20011, 3)], [(3, 20), (6000, 1)],
                                  [(900, 1), (2100, 4), (64, 2), (8190, 2)]],
                         ids=lambda rows: f"{len(rows)}x{rows[-1]}")
@pytest.mark.parametrize("kv_heads, group, dim", [(8, 4, 128), (1, 7, 64)])
def test_few_items_give_the_same_bits(w4lib, rows, kv_heads, group, dim):
    args = make(rows, kv_heads, group, dim, 16, torch.float16, seed=len(rows))
    want, want_lse = w4.paged_chunk_attention(*args, return_lse=True)
    differs = torch.zeros((), dtype=torch.bool, device="cuda")
    for _ in range(CALLS):
        out, lse = w4.paged_chunk_attention(*args, return_lse=True)
        differs |= (out.view(torch.int16) != want.view(torch.int16)).any()
        differs |= (lse != want_lse).any()
    assert not differs.item()
    assert w4.device_status() == 0
