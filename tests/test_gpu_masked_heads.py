"""kvq_paged_decode_window and kvq_paged_decode_tree over several KV heads: units that hold up to four
heads side by side, last groups of fewer, and what one head's cache rows do to the others (nothing)."""
import pytest
import torch

import fp8_paged_kv_kvq_gb300 as kvq
import oracle.masked as plain
from test_gpu_masked import (SCALE, assert_close, check_tree, check_window, make, on_gpu, queries,
                             random_mask, tree, window, words_of)

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


def spoil(c, slot, h, how):
    """A row of one head: one NaN code, or what the store makes of a row with a NaN."""
    if how == "code":
        c["v_codes"][slot, h, 5] = 0x7F
    else:
        for x in ("k", "v"):
            c[x + "_codes"][slot, h] = 0x7F
            c[x + "_scales"][slot, h] = float("nan")


@pytest.mark.parametrize("how", ["code", "row"])
@pytest.mark.parametrize("G,R", [(1, 1), (4, 2), (4, 8), (3, 11), (4, 16), (5, 13), (4, 40)])
@pytest.mark.parametrize("H", [2, 3, 4, 5, 8])
def test_what_one_head_holds_does_not_reach_the_others(H, G, R, how):
    """A row of one head of a context token that every row sees, in a chunk that every row sees whole
    (token 70 and 201) and in one that some rows do not (a drafted token): its own head's rows that see
    it become NaN, all other rows are what they were (bit for bit where only a code
    changed; a scale can move the power of two that a unit's weights are held over, which moves
    roundings)."""
    bs, lens, h = 16, [300 + R, R, 41 + R], H - 1 if H != 4 else 2
    c, tables = make(lens, H, bs, 211 + H)
    q = queries(len(lens) * R, H * G, 13 * R + G)
    bits = torch.zeros(len(lens), R, -(-R // 32) * 32, dtype=torch.int64)
    for i in range(R):
        bits[:, i, i] = 1
        bits[:, i, i % 2:i:2] = 1
    mask = words_of(bits)
    rules = (plain.window_rule(10 ** 6, 0), plain.tree_rule(mask))
    want = [plain.attention(c, q, tables, lens, R, SCALE, rule) for rule in rules]

    def calls(cache):
        return window(cache, q, tables, lens, 10 ** 6, 0, R), tree(cache, q, mask, tables, lens, R)

    clean = calls(on_gpu(c))
    for j, request in ((70, 0), (201, 0), (300 + R - 1, 0), (41, 2)):
        spoiled = {n: x.clone() if n != "block_size" else x for n, x in c.items()}
        spoil(spoiled, slot_of(tables, request, j, bs), h, how)
        for got, was, ref, rule in zip(calls(on_gpu(spoiled)), clean, want, rules):
            sees = rule(lens[request], R, request)[:, j]
            hit = torch.zeros(len(lens) * R, H, dtype=torch.bool)
            hit[request * R:(request + 1) * R, h] = sees
            rows, others = heads_of(got, H), ~hit
            if how == "code":
                assert torch.equal(rows[others], heads_of(was, H)[others])
                assert bool(torch.isnan(rows[hit][..., 5]).all())
            else:
                assert_close(rows[others], tuple(x.view(*rows.shape[:3], -1)[others] for x in ref), lens)
                assert bool(torch.isnan(rows[hit]).all())


@pytest.mark.parametrize("H,G", [(4, 4), (5, 2), (2, 16)])
def test_nan_of_one_of_many_units(H, G):
    """Blocks with many units of one chunk and of several, one request and head of them with a NaN: the
    units before and after it are what they were."""
    bs = 16
    lens = [(32, 64, 1, 100)[i % 4] for i in range(900)]
    c, tables = make(lens, H, bs, 311)
    q = queries(len(lens), H * G, 311)
    clean = heads_of(window(on_gpu(c), q, tables, lens, 10 ** 6, 0, 1), H)
    for request, j, h in ((0, 3, 0), (4, 31, H - 1), (441, 40, 1), (640, 0, H - 1), (899, 99, 0), (898, 0, 1)):
        codes = c["v_codes"].clone()
        c["v_codes"][slot_of(tables, request, j, bs), h, 5] = 0xFF
        got = heads_of(window(on_gpu(c), q, tables, lens, 10 ** 6, 0, 1), H)
        c["v_codes"] = codes
        hit = torch.zeros(len(lens), H, dtype=torch.bool)
        hit[request, h] = True
        assert torch.equal(got[~hit], clean[~hit])
        assert bool(torch.isnan(got[hit][..., 5]).all())


def test_nan_in_pieces_of_a_split_unit():
    """One request whose chunks are shared out over the whole GPU and joined."""
    H, bs, lens = 6, 16, [9000]
    c, tables = make(lens, H, bs, 401)
    q = queries(3, 4 * H, 401)
    clean = heads_of(window(on_gpu(c), q, tables, lens, 10 ** 6, 0, 3), H)
    for j, h in ((0, 0), (4321, 2), (8000, 5), (8996, 4)):
        codes = c["v_codes"].clone()
        c["v_codes"][slot_of(tables, 0, j, bs), h, 5] = 0x7F
        got = heads_of(window(on_gpu(c), q, tables, lens, 10 ** 6, 0, 3), H)
        c["v_codes"] = codes
        other = torch.arange(H) != h
        assert torch.equal(got[:, other], clean[:, other])
        assert bool(torch.isnan(got[:, h, :, 5]).all())


@pytest.mark.parametrize("w,sinks", [(2 ** 32 + 5, 0), (2 ** 40, 2 ** 32 + 1), (10 ** 12, 10 ** 10), (7, 2 ** 33)])
def test_windows_and_sinks_beyond_32_bits(w, sinks):
    """Numbers that mean every token, whatever their lower 32 bits are."""
    lens, H, R = [200, 33], 2, 2
    c, tables = make(lens, H, 16, 601)
    q = queries(len(lens) * R, 4, 601)
    assert_close(window(on_gpu(c), q, tables, lens, w, sinks, R),
                 plain.attention(c, q, tables, lens, R, SCALE, plain.window_rule(10 ** 6, 0)), lens)


@pytest.mark.parametrize("H,G,R", [(2, 5, 40), (3, 4, 40), (5, 2, 65), (4, 8, 64), (2, 1, 300), (3, 16, 9), (2, 64, 2)])
def test_row_tiles_of_several_heads(H, G, R):
    """From 128 stacked rows on: units of one or two row tiles, a unit per head and tile."""
    lens = [R + 500, R, 0, R + 70]
    check_window(lens, H, H * G, R, 200, 5, seed=H * R)
    check_window(lens, H, H * G, R, 33, 0, bs=64, seed=H + R)
    check_tree(lens, H, H * G, R, seed=G * R)


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("H,G,R", [(1, 4, 20), (3, 4, 32), (2, 8, 17), (2, 4, 70), (1, 16, 33)])
def test_trees_over_large_pages(bs, H, G, R):
    """Trees of one head a unit, whose copies bring whole pages (of at most 128 tokens): pages that end
    inside a chunk, at its end and behind it, and contexts that end in each of their parts."""
    for lens in ([R + 4 * bs, R + bs - 1, R], [R + 3 * bs + 1, 700 + R, R + 2 * bs + 17], [R + 1, R + 127, R + 128]):
        check_tree(lens, H, H * G, R, bs=bs, seed=bs + R + len(lens))


@pytest.mark.parametrize("seed", range(12))
def test_small_calls_of_all_shapes(seed):
    """Random heads, groups, rows, pages and lengths, new tensors each time, each call twice."""
    g = torch.Generator().manual_seed(700 + seed)

    def one(*values):
        return values[int(torch.randint(0, len(values), (1,), generator=g))]

    for i in range(12):
        H, G, R, n = one(1, 2, 3, 4, 5, 6, 7, 9), one(1, 2, 3, 4, 7), one(1, 1, 2, 3, 5, 9, 10, 17, 40), one(1, 2, 3)
        bs, w, sinks = one(16, 32, 64), one(1, 16, 50, 1000), one(0, 1, 3, 40)
        lens = [one(0, R - 1, R, R + 31, R + int(torch.randint(0, 300, (1,), generator=g))) for _ in range(n)]
        c, tables = make(lens, H, bs, 1000 * seed + i)
        q, mask, most = queries(n * R, H * G, i), random_mask(n, R, i), max(max(lens), 1)
        cache = on_gpu(c)
        for call, rule in ((lambda: window(cache, q, tables, lens, w, sinks, R, most=most), plain.window_rule(w, sinks)),
                           (lambda: tree(cache, q, mask, tables, lens, R, most=most), plain.tree_rule(mask))):
            got = call()
            assert_close(got, plain.attention(c, q, tables, lens, R, SCALE, rule), lens)
            assert torch.equal(got, call())
