"""kvq_paged_decode_window and kvq_paged_decode_tree over several KV heads: units that hold up to four
heads side by side, last groups of fewer, and what one head's cache rows do to the others (nothing)."""
import pytest
import torch

import fp8_paged_kv_kvq_gb300 as kvq
import oracle.masked as plain
from test_gpu_masked import (SCALE, assert_close, check_tree, check_window, make, on_gpu, queries, tree,
                             window)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [5, 6, 7, 9, 10, 11])
@pytest.mark.parametrize("G,R", [(1, 1), (4, 5), (2, 25)])
def test_last_groups_of_fewer_heads(H, G, R):
    """One to three heads behind the groups of four (two): keys of pages next to the planes' ends."""
    lens = [R + 300, R, 0, R + 33]
    check_window(lens, H, H * G, R, 120, 4, seed=H + R, spare=0)
    check_tree(lens, H, H * G, R, seed=H * R, spare=0)


@pytest.mark.parametrize("H", [1, 3, 5, 7])
def test_last_groups_at_the_end_of_memory(H):
    """The planes side by side, values first, at the end of their allocation."""
    lens, R = [100, 31], 3
    c, tables = make(lens, H, 16, 7 + H, spare=0)
    q = queries(len(lens) * R, 2 * H, 7)
    n = c["k_codes"].numel()
    memory = torch.empty(2 * n, dtype=torch.uint8, device="cuda")
    k, v = memory[n:].view(c["k_codes"].shape), memory[:n].view(c["k_codes"].shape)
    k.copy_(c["k_codes"])
    v.copy_(c["v_codes"])
    cache = kvq.Cache(k, v, c["k_scales"].cuda(), c["v_scales"].cuda(), 16)
    assert_close(window(cache, q, tables, lens, 50, 3, R),
                 plain.attention(c, q, tables, lens, R, SCALE, plain.window_rule(50, 3)), lens)
    mask = torch.tensor([[[0b001], [0b011], [0b101]]] * 2, dtype=torch.int32)
    assert_close(tree(cache, q, mask, tables, lens, R),
                 plain.attention(c, q, tables, lens, R, SCALE, plain.tree_rule(mask)), lens)
