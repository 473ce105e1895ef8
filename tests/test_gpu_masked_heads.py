"""kvq_paged_decode_window and kvq_paged_decode_tree over several KV heads: units that hold up to four
heads side by side, last groups of fewer, and what one head's cache rows do to the others (nothing)."""
import pytest
import torch

import fp8_paged_kv_kvq_gb300 as kvq
import oracle.masked as plain
from test_gpu_masked import (SCALE, assert_close, check_tree, check_window, make, on_gpu, queries, tree,
                             window, words_of)

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


def slot_of(tables, r, j, bs):
    return int(tables[r, j // bs]) * bs + j % bs


def heads_of(got, H):
    """[rows, H, G, 128]"""
    return got.cpu().view(got.shape[0], H, -1, 128)


@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("H,G,R", [(1, 1, 1), (1, 4, 2), (3, 5, 3), (4, 4, 8), (5, 4, 2), (2, 3, 11), (2, 4, 16), (1, 5, 13),
                                   (2, 5, 20), (1, 4, 40), (2, 5, 64)])
def test_value_scales_that_are_not_finite(H, G, R, value):
    """One such scale, of a token that every row sees, in the first chunk, in later ones that every row
    sees whole and in the last: no row that sees it is finite, all others (of other heads, requests and
    branches) are right."""
    bs, lens, h = 16, [300 + R, R, 141 + R], H // 2
    c, tables = make(lens, H, bs, 511 + H)
    q = queries(len(lens) * R, H * G, 13 * R + G)
    bits = torch.zeros(len(lens), R, -(-R // 32) * 32, dtype=torch.int64)
    for i in range(R):
        bits[:, i, i] = 1
        bits[:, i, i % 2:i:2] = 1
    mask = words_of(bits)
    rules = (plain.window_rule(10 ** 6, 0), plain.tree_rule(mask))
    want = [plain.attention(c, q, tables, lens, R, SCALE, rule) for rule in rules]
    for j, request in ((0, 0), (70, 0), (201, 2), (300 + R - 1, 0)):
        j = min(j, lens[request] - 1)
        was = c["v_scales"].clone()
        c["v_scales"][slot_of(tables, request, j, bs), h] = value
        cache = on_gpu(c)
        c["v_scales"] = was
        outs = (window(cache, q, tables, lens, 10 ** 6, 0, R), tree(cache, q, mask, tables, lens, R))
        for got, ref, rule in zip(outs, want, rules):
            hit = torch.zeros(len(lens) * R, H, dtype=torch.bool)
            hit[request * R:(request + 1) * R, h] = rule(lens[request], R, request)[:, j]
            rows = heads_of(got, H)
            assert_close(rows[~hit], tuple(x.view(*rows.shape[:3], -1)[~hit] for x in ref), lens)
            assert bool(hit.any()) and not bool(torch.isfinite(rows[hit]).any())
