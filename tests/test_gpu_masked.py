"""kvq_paged_decode_window and kvq_paged_decode_tree on the GPU against fp64 attention over the
same cache (oracle/masked.py).

Tolerance.  Of an output o = sum_j w_j v_j the kernel rounds: the output to bf16 (2^-8 |o|); every
probability times its value scale to f16 for the product (2^-11 sum_j w_j |v_j|; the sum's
denominator is not rounded, the value codes are exact in f16); those below the f16 normal range, at
a scale of at most 4 times the largest value scale seen and under a reference that the row's largest
probability is not below, are off by 2^-25 each, times 448 times that scale, which is at most 4 and
with the codec's rounding 4.3 times the largest |v| seen: together at most L 2^-22 max |v|; the score
of 256 binary32 additions (two pieces of the query) and its scaling, an absolute error of at most
260 2^-23 max_j sm_scale sum_d |q_d k_jd|, and the query elements below 2^-9 of their row's largest
(2^-17 of it each), 2^-17 sm_scale max |q_d| max_j sum_d |k_jd|: together e, which moves numerator and
denominator by a relative e each; the exponentials, 2^-20 each; and the two sums of up to L terms, a
unit in the last place per addition, L 2^-22 together.  In all
    |err| <= 2^-8 |o| + (2^-11 + 2 e + 2^-19 + L 2^-22) sum_j w_j |v_j| + L 2^-22 max |v|."""
import pytest
import torch

import fp8_paged_kv_kvq_gb300 as kvq
import oracle.masked as plain

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5
F8 = torch.float8_e4m3fn


def make(lens, H, bs, seed, spare=3, width=0, k_spread=1.0, v_spread=None):
    """A cache of N(0, 1) rows with every request's pages in random order; CPU copies beside it.
    v_spread: per-position factors of the value rows (positions of all requests)."""
    g = torch.Generator().manual_seed(seed)
    pages = [-(-n // bs) for n in lens]
    total = sum(pages) + spare
    order = torch.randperm(total, generator=g).to(torch.int32)
    width = max(max(pages, default=0), 1) + width
    tables = torch.full((len(lens), width), -1, dtype=torch.int32)
    at = 0
    for row, p in zip(tables, pages):
        row[:p] = order[at:at + p]
        at += p
    c = dict(block_size=bs)
    for name, f in (("k", k_spread), ("v", 1.0)):
        x = torch.randn(total * bs, H, 128, generator=g) * f
        if name == "v" and v_spread is not None:
            for row, n in zip(tables, lens):
                j = torch.arange(n)
                x[row[j // bs].long() * bs + j % bs] *= v_spread[:n, None, None]
        s = x.abs().amax(-1) / 448
        c[name + "_codes"] = torch.where(s[..., None] > 0, x / s[..., None], torch.zeros_like(x)).to(F8).view(torch.uint8)
        c[name + "_scales"] = s
    return c, tables


def on_gpu(c):
    return kvq.Cache(c["k_codes"].cuda(), c["v_codes"].cuda(), c["k_scales"].cuda(),
                     c["v_scales"].cuda(), c["block_size"])


def queries(n, hq, seed, spread=1.5):
    g = torch.Generator().manual_seed(seed + 77)
    return (torch.randn(n, hq, 128, generator=g) * spread).to(torch.bfloat16)


def random_mask(n, r, seed):
    g = torch.Generator().manual_seed(seed + 5)
    bits = torch.zeros(n, r, -(-r // 32) * 32, dtype=torch.int64)
    for i in range(r):
        for a in range(n):
            parent = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
            if parent >= 0:
                bits[a, i] = bits[a, parent]
            bits[a, i, i] = 1
    return words_of(bits)


def words_of(bits):
    w = (bits.reshape(*bits.shape[:-1], -1, 32).long() << torch.arange(32)).sum(-1)
    return torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)


def assert_close(got, want, lens):
    ref, mag, big, dot, peak = want
    n = max(max(lens), 1)
    e = 260 * 2.0 ** -23 * dot + 2.0 ** -17 * peak
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -11 + 2 * e + 2.0 ** -19 + n * 2.0 ** -22) * mag + n * 2.0 ** -22 * big
    got = got.cpu().double()
    assert bool(torch.isfinite(got).all())
    err = (got - ref).abs()
    assert bool((err[tol == 0] == 0).all())                 # rows that see nothing are zero
    worst = float((err / tol.clamp(min=1e-300)).max()) if err.numel() else 0.0
    print(f"worst |err| / bound {worst:.3f}")
    assert worst <= 1.0


def window(cache, q, tables, lens, w, sinks, R, err=0, most=None, scale=SCALE, **kw):
    e = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = kvq.paged_decode_window(cache, q.cuda(), tables.cuda(),
                                  torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                  max(lens) if most is None else most, w, scale, num_sinks=sinks,
                                  rows_per_request=R, err_flags=e, **kw)
    torch.cuda.synchronize()
    assert int(e) == err
    return out


def tree(cache, q, mask, tables, lens, R, err=0, most=None, scale=SCALE, **kw):
    e = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = kvq.paged_decode_tree(cache, q.cuda(), mask.cuda(), tables.cuda(),
                                torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                max(lens) if most is None else most, scale, R, err_flags=e, **kw)
    torch.cuda.synchronize()
    assert int(e) == err
    return out


def check_window(lens, H, hq, R, w, sinks, bs=16, seed=0, **kw):
    c, tables = make(lens, H, bs, seed, **kw)
    q = queries(len(lens) * R, hq, seed)
    got = window(on_gpu(c), q, tables, lens, w, sinks, R)
    assert_close(got, plain.attention(c, q, tables, lens, R, SCALE, plain.window_rule(w, sinks)), lens)


def check_tree(lens, H, hq, R, bs=16, seed=0, mask=None, **kw):
    c, tables = make(lens, H, bs, seed, **kw)
    q = queries(len(lens) * R, hq, seed)
    mask = random_mask(len(lens), R, seed) if mask is None else mask
    got = tree(on_gpu(c), q, mask, tables, lens, R)
    assert_close(got, plain.attention(c, q, tables, lens, R, SCALE, plain.tree_rule(mask)), lens)


LENS = [[1], [2], [16], [17], [127], [128], [129], [255, 256, 257], [0, 5, 0, 0, 130, 0], [31, 400, 64], [1000]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("w,sinks", [(1, 0), (1, 1), (7, 4), (100, 0), (128, 16), (10000, 3)])
def test_window_one_row(lens, w, sinks):
    check_window(lens, 2, 8, 1, w, sinks, seed=sum(lens) + w)


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("hq,H", [(32, 8), (3, 3), (7, 1), (16, 1)])
def test_tree_lengths(lens, hq, H):
    check_tree(lens, H, hq, 5, seed=sum(lens) + hq)


@pytest.mark.parametrize("hq,H", [(1, 1), (2, 1), (3, 3), (10, 2), (12, 4), (14, 2), (32, 2), (64, 1), (40, 5)])
def test_head_layouts(hq, H):
    check_window([200, 333], H, hq, 1, 150, 4, seed=hq)
    check_tree([200, 333], H, hq, 6, seed=hq)


@pytest.mark.parametrize("R", [2, 3, 8, 9, 31, 32, 33, 64, 65, 100, 129, 300])
def test_window_rows(R):
    """From two rows to several row tiles, the window shorter and longer than the rows."""
    for w, sinks in ((20, 2), (150, 33)):
        check_window([R, R + 1, 500 + R], 1, 4, R, w, sinks, seed=R + w)


@pytest.mark.parametrize("R", [1, 2, 4, 8, 9, 16, 31, 32, 33, 64, 65, 96])
def test_tree_rows(R):
    check_tree([R, R + 1, 500 + R], 1, 4, R, seed=R)


def test_tree_many_nodes():
    g = torch.Generator().manual_seed(3)
    bits = (torch.rand(1, 200, 224, generator=g) < 0.3).long()
    check_tree([700], 1, 2, 200, mask=words_of(bits))


@pytest.mark.parametrize("bs", [16, 32, 64, 128, 256, 1024])
def test_pages(bs):
    lens = [bs - 1, bs, bs + 1, 3 * bs + 5]
    check_window(lens, 2, 4, 3, 2 * bs, 5, bs=bs, seed=bs)
    check_tree([n + 6 for n in lens], 2, 4, 6, bs=bs, seed=bs)


@pytest.mark.parametrize("sinks", [0, 1, 15, 16, 17, 127, 128, 129, 300, 5000])
def test_sinks(sinks):
    """Sinks apart from the window, next to it, overlapping it and beyond the context."""
    for w in (1, 64, 400):
        check_window([450, 20], 1, 4, 1, w, sinks, seed=sinks + w)
    check_window([450, 20], 1, 4, 7, 64, sinks, seed=sinks)


def test_rows_before_the_sequence_are_zero():
    check_window([3, 0, 1], 2, 8, 4, 5, 1, seed=1)
    check_tree([3, 0, 1], 2, 8, 4, seed=1)
    check_window([40], 1, 4, 64, 5, 1, seed=2)


def test_masks_that_leave_rows_empty():
    mask = torch.zeros(2, 4, 1, dtype=torch.int32)
    mask[0, 1] = 0b0010
    mask[1, 3] = 0b0110
    check_tree([4, 4], 2, 8, 4, mask=mask, seed=4)          # no context: rows without bits see nothing
    check_tree([4, 20], 2, 8, 4, mask=mask, seed=5)
    check_tree([40, 20], 2, 8, 4, mask=torch.full((2, 4, 1), -1, dtype=torch.int32), seed=6)   # later nodes too


def test_split_over_many_blocks():
    """One request and head: its keys are shared out over the whole GPU and joined."""
    check_window([9000], 1, 4, 1, 8500, 4, seed=8)
    check_tree([9001], 1, 8, 4, seed=9)
    check_tree([6000], 1, 4, 40, seed=10)
    check_tree([5000], 1, 4, 70, seed=11)


def test_many_requests():
    lens = [(7 * i) % 50 for i in range(2100)]
    check_window(lens, 1, 2, 1, 16, 2, seed=12)
    check_tree([n + 3 if n else 0 for n in lens], 1, 1, 3, seed=13)


def test_idle_requests():
    check_window([0, 0, 0], 2, 8, 1, 5, 1)
    check_window([0] * 40 + [77], 2, 8, 2, 50, 1)


def test_evicted_pages_are_not_read():
    """Table entries outside sinks and window hold anything; the pages they held are poisoned."""
    lens, R, w, sinks, bs = [900, 333, 64], 3, 100, 20, 16
    c, tables = make(lens, 2, bs, 21)
    q = queries(len(lens) * R, 8, 21)
    want = plain.attention(c, q, tables, lens, R, SCALE, plain.window_rule(w, sinks))
    for r, n in enumerate(lens):
        for p in range(-(-n // bs)):
            if p * bs >= sinks and (p + 1) * bs <= n - R + 1 - w:
                slot = int(tables[r, p]) * bs
                for x in ("k", "v"):
                    c[x + "_codes"][slot:slot + bs] = 0x7F
                    c[x + "_scales"][slot:slot + bs] = float("nan")
                tables[r, p] = (-1, 1 << 30, -2 ** 31)[p % 3]
    assert_close(window(on_gpu(c), q, tables, lens, w, sinks, R), want, lens)


@pytest.mark.parametrize("poison", ["nan", "inf", "huge"])
@pytest.mark.parametrize("R", [3, 40])
def test_unseen_tokens_do_not_reach_rows(poison, R):
    """NaN, infinities and huge values in slots that share pages and tiles with seen ones: behind
    the context, between sinks and window, and in drafted tokens of other branches."""
    bs, lens = 32, [75 + R, 301 + R]
    value = dict(nan=float("nan"), inf=float("inf"), huge=1e30)[poison]

    def spoil(c, slot):
        for x in ("k", "v"):
            c[x + "_codes"][slot] = 0x7F if poison == "nan" else 0x7E
            c[x + "_scales"][slot] = value

    w, sinks = 40, 3
    c, tables = make(lens, 1, bs, 31)
    q = queries(len(lens) * R, 4, 31)
    want = plain.attention(c, q, tables, lens, R, SCALE, plain.window_rule(w, sinks))
    for r, n in enumerate(lens):
        for j in list(range(sinks, n - R + 1 - w)) + list(range(n, -(-n // bs) * bs)):
            spoil(c, int(tables[r, j // bs]) * bs + j % bs)
    assert_close(window(on_gpu(c), q, tables, lens, w, sinks, R), want, lens)

    # every second node is on one branch; the others' rows are poisoned, and only their own
    # queries see them
    c, tables = make(lens, 1, bs, 32)
    bits = torch.zeros(2, R, -(-R // 32) * 32, dtype=torch.int64)
    for i in range(R):
        bits[:, i, i] = 1
        bits[:, i, i % 2:i:2] = 1
    mask = words_of(bits)
    want = plain.attention(c, q, tables, lens, R, SCALE, plain.tree_rule(mask))
    for r, n in enumerate(lens):
        for b in range(1, R, 2):
            spoil(c, int(tables[r, (n - R + b) // bs]) * bs + (n - R + b) % bs)
    got = tree(on_gpu(c), q, mask, tables, lens, R).cpu()
    clean = torch.arange(2 * R) % R % 2 == 0
    assert_close(got[clean], tuple(x[clean] for x in want), lens)
    if poison != "huge":
        assert bool((~torch.isfinite(got[~clean])).any(dim=-1).all())
    # and a window's own: a poisoned token is seen by the rows that reach it and by no others
    if R < 40:
        return
    c, tables = make(lens, 1, bs, 33)
    n = lens[1]
    at = n - R + 1 - 20                                    # the last token outside row 20's window
    want = plain.attention(c, q, tables, lens, R, SCALE, plain.window_rule(w, sinks))
    reach = at + w - (n - R)                               # rows below see it
    assert 0 < reach < R
    spoil(c, int(tables[1, at // bs]) * bs + at % bs)
    got = window(on_gpu(c), q, tables, lens, w, sinks, R).cpu()
    clean = torch.cat([torch.ones(R, dtype=torch.bool), torch.arange(R) >= reach])
    assert_close(got[clean], tuple(x[clean] for x in want), lens)


def test_value_code_of_nan():
    lens, R, bs = [140], 4, 16
    c, tables = make(lens, 1, bs, 41)
    q = queries(R, 4, 41)
    mask = torch.tensor([[[0b0001], [0b0011], [0b0101], [0b1011]]], dtype=torch.int32)
    j = 140 - 4 + 1                                        # node 1: seen by rows 1 and 3
    c["v_codes"][int(tables[0, j // bs]) * bs + j % bs, 0, 5] = 0x7F
    got = tree(on_gpu(c), q, mask, tables, lens, R).cpu()
    assert bool(torch.isfinite(got[[0, 2]]).all()) and bool(torch.isnan(got[[1, 3], :, 5]).all())


@pytest.mark.parametrize("R,hq", [(1, 4), (8, 4), (40, 4), (80, 8)])
def test_references_move(R, hq):
    """Keys and values that grow along the context: later tokens outweigh all before them, and
    value scales climb over many binades."""
    n = 700 + R
    up = torch.logspace(-3, 3, n)
    check_tree([n], 1, hq, R, seed=51, v_spread=up)
    check_window([n], 1, hq, R, 300, 5, seed=52, v_spread=up.flip(0))
    c, tables = make([n], 1, 16, 53)
    j = torch.arange(n)
    slot = tables[0, j // 16].long() * 16 + j % 16
    q = queries(R, hq, 53)
    c["k_scales"][slot] *= torch.linspace(0.01, 12.0, n)[:, None]     # scores of a growing spread
    for rule, got in ((plain.window_rule(500, 7), window(on_gpu(c), q, tables, [n], 500, 7, R)),
                      (plain.window_rule(10 ** 6, 0), window(on_gpu(c), q, tables, [n], 10 ** 6, 0, R))):
        assert_close(got, plain.attention(c, q, tables, [n], R, SCALE, rule), [n])


def test_scores_far_below_the_first_ones():
    """Rows whose early tokens dominate, and rows whose scores are all far below zero."""
    n = 600
    c, tables = make([n], 1, 16, 61)
    q = queries(1, 4, 61)
    j = torch.arange(n)
    slot = tables[0, j // 16].long() * 16 + j % 16
    c["k_scales"][slot] *= torch.linspace(20.0, 0.01, n)[:, None]
    got = window(on_gpu(c), q, tables, [n], 10 ** 6, 0, 1)
    assert_close(got, plain.attention(c, q, tables, [n], 1, SCALE, plain.window_rule(10 ** 6, 0)), [n])
    c["k_codes"][:] = torch.full_like(c["k_codes"], 0x40)              # every score the same, far below 0
    c["k_scales"][:] = 1.0
    q = torch.full_like(q, -3.0)
    got = window(on_gpu(c), q, tables, [n], 300, 5, 1)
    assert_close(got, plain.attention(c, q, tables, [n], 1, SCALE, plain.window_rule(300, 5)), [n])


def test_zero_rows_and_scales():
    c, tables = make([300], 2, 16, 71)
    c["k_scales"][:] = 0
    c["v_scales"][::2] = 0
    q = queries(5, 8, 71)
    got = window(on_gpu(c), q, tables, [300], 200, 3, 5)
    assert_close(got, plain.attention(c, q, tables, [300], 5, SCALE, plain.window_rule(200, 3)), [300])
    got = window(on_gpu(c), torch.zeros_like(q), tables, [300], 200, 3, 5)
    assert_close(got, plain.attention(c, torch.zeros_like(q), tables, [300], 5, SCALE,
                                      plain.window_rule(200, 3)), [300])
    c["v_scales"][:] = 0
    assert bool((window(on_gpu(c), q, tables, [300], 200, 3, 5) == 0).all())


@pytest.mark.parametrize("scale", [-0.05, 0.0, 1e-3])
def test_scales_of_the_softmax(scale):
    c, tables = make([260], 1, 16, 73)
    q = queries(3, 4, 73)
    got = window(on_gpu(c), q, tables, [260], 100, 4, 3, scale=scale)
    assert_close(got, plain.attention(c, q, tables, [260], 3, scale, plain.window_rule(100, 4)), [260])


def test_bad_pages_and_lengths_are_flagged():
    """Device data that is out of range is reported, never read; other requests stay exact."""
    lens = [200, 210, 220]
    c, tables = make(lens, 2, 16, 81)
    q = queries(3, 8, 81)
    want = plain.attention(c, q, tables, lens, 1, SCALE, plain.window_rule(64, 4))
    bad = tables.clone()
    bad[1, 12] = 10 ** 9
    got = window(on_gpu(c), q, bad, lens, 64, 4, 1, err=kvq.ERRF_BLOCK_RANGE)
    keep = [0, 2]
    assert_close(got[keep], tuple(x[keep] for x in want), lens)
    bad[1, 12] = -5
    window(on_gpu(c), q, bad, lens, 64, 4, 1, err=kvq.ERRF_BLOCK_RANGE)
    got = window(on_gpu(c), q, tables, [200, -3, 220], 64, 4, 1, err=kvq.ERRF_CONTEXT_RANGE)
    assert_close(got[keep], tuple(x[keep] for x in want), lens)
    assert bool((got[1] == 0).all())
    got = window(on_gpu(c), q, tables, [200, 10 ** 9, 220], 64, 4, 1, err=kvq.ERRF_CONTEXT_RANGE, most=220)
    assert_close(got[keep], tuple(x[keep] for x in want), lens)


def test_scale_planes_of_any_alignment():
    c, tables = make([100, 50], 3, 16, 91)
    q = queries(2 * 2, 6, 91)
    cache = on_gpu(c)
    for name in ("k_scales", "v_scales"):
        t = getattr(cache, name)
        odd = torch.zeros(t.numel() + 1, device="cuda")[1:].view(t.shape)
        odd.copy_(t)
        setattr(cache, name, odd)
    got = window(cache, q, tables, [100, 50], 64, 4, 2)
    assert_close(got, plain.attention(c, q, tables, [100, 50], 2, SCALE, plain.window_rule(64, 4)), [100])


def test_wide_window_agrees_with_paged_decode():
    lens = [777, 1200]
    c, tables = make(lens, 4, 16, 95)
    q = queries(2 * 4, 16, 95)
    cache = on_gpu(c)
    got = window(cache, q, tables, lens, 10 ** 6, 0, 4)
    ref = kvq.paged_decode(cache, q.cuda(), tables.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                           1200, SCALE, rows_per_request=4)
    assert float((got.float() - ref.float()).abs().max()) <= 2 * 1e-2


def test_same_results_every_time():
    lens = [3000, 100, 2500]
    c, tables = make(lens, 2, 16, 97)
    cache = on_gpu(c)
    for R in (2, 40):
        q, mask = queries(3 * R, 8, 97), random_mask(3, R, 97)
        first = tree(cache, q, mask, tables, lens, R)
        for _ in range(3):
            assert torch.equal(first, tree(cache, q, mask, tables, lens, R))


def test_graphs_that_share_a_workspace_and_streams():
    """A window's and a tree's captured call with one workspace, replayed in turn on new lengths and
    queries; and a call on a stream of its own."""
    lens, R = [640, 1500], 4
    c, tables = make([1500, 1500], 2, 16, 99)          # (pages for every length below)
    cache = on_gpu(c)
    q = queries(2 * R, 8, 99).cuda()
    mask = random_mask(2, R, 99)
    tb, mk, cl = tables.cuda(), mask.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    size = max(kvq.paged_decode_window_workspace_size(2, R, 8, 2, 128, 16, 1500, 300, 4),
               kvq.paged_decode_tree_workspace_size(2, R, 8, 2, 128, 16, 1500), 1)
    ws = torch.randint(0, 256, (size,), dtype=torch.uint8, device="cuda")
    outs = [torch.full_like(q, 5.0) for _ in range(2)]
    calls = [lambda s=None: kvq.paged_decode_window(cache, q, tb, cl, 1500, 300, SCALE, num_sinks=4,
                                                    rows_per_request=R, out=outs[0], workspace=ws, stream=s),
             lambda s=None: kvq.paged_decode_tree(cache, q, mk, tb, cl, 1500, SCALE, R, out=outs[1],
                                                  workspace=ws, stream=s)]
    graphs = []
    for call in calls:
        call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call()
        graphs.append(g)
    rules = (plain.window_rule(300, 4), plain.tree_rule(mask))
    for new in (lens, [1200, 700], [R, 0]):
        cl.copy_(torch.tensor(new, dtype=torch.int32))
        q.copy_(queries(2 * R, 8, sum(new)))
        for _ in range(2):
            for g in graphs:
                g.replay()
        torch.cuda.synchronize()
        for out, rule in zip(outs, rules):
            assert_close(out, plain.attention(c, q.cpu(), tables, new, R, SCALE, rule), new)
    side = torch.cuda.Stream()
    for out, call, rule in zip(outs, calls, rules):
        out.fill_(3.0)
        side.wait_stream(torch.cuda.current_stream())
        call(side)
        side.synchronize()
        assert_close(out, plain.attention(c, q.cpu(), tables, [R, 0], R, SCALE, rule), [R])


def test_rows_around_the_output_stay():
    c, tables = make([50, 70], 2, 16, 103)
    q = queries(4, 8, 103)
    big = torch.full((8, 8, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    window(on_gpu(c), q, tables, [50, 70], 20, 2, 2, out=big[2:6])
    assert bool((big[:2] == 9).all()) and bool((big[6:] == 9).all()) and not bool((big[2:6] == 9).any())


def test_no_requests():
    c, tables = make([50], 2, 16, 105)
    q = torch.zeros(0, 8, 128, dtype=torch.bfloat16)
    out = kvq.paged_decode_window(on_gpu(c), q.cuda(), tables[:0].cuda(),
                                  torch.zeros(0, dtype=torch.int32, device="cuda"), 50, 20, SCALE)
    assert out.shape == (0, 8, 128)


def test_more_chunks_than_16_bits_count():
    # 1,024 requests of 2^20 tokens over the same 64 pages: over 100,000 chunks a block and chain.
    # Keys of score 0 and integers as values: weights of 1 and all sums (below 2^24) are exact, so
    # that only the division, the pieces' joining (under 32 roundings) and bf16 round.
    n, most, bs, pages = 1024, 1 << 20, 64, 64
    g = torch.Generator().manual_seed(3)
    v = torch.randint(0, 8, (pages * bs, 1, 128), generator=g).float()
    c = dict(block_size=bs, v_codes=v.to(F8).view(torch.uint8), v_scales=torch.ones(pages * bs, 1),
             k_codes=torch.randn(pages * bs, 1, 128, generator=g).to(F8).view(torch.uint8),
             k_scales=torch.ones(pages * bs, 1))
    order = torch.randperm(pages, generator=g).to(torch.int32)
    tables = order.repeat(most // bs // pages)[None].cuda().expand(n, -1).contiguous()
    got = window(on_gpu(c), torch.zeros(n, 1, 128, dtype=torch.bfloat16), tables, [most] * n, most, 0, 1)
    want = v.double().mean(0)
    assert bool(((got.cpu().double() - want).abs() <= (2.0 ** -8 + 2.0 ** -19) * want).all())


@pytest.mark.parametrize("H", [1, 2, 3, 5])
def test_few_heads_in_planes_far_apart(H):
    # the planes' copies stay in their planes: fewer heads than a unit has places, a gap of
    # other memory between the planes, the values' plane in front of the keys'
    lens = [123, 1, 40]
    c, tables = make(lens, H, 16, 107 + H)
    q = queries(3, H, 107)
    n = c["k_codes"].numel()
    memory = torch.empty(1700 << 20, dtype=torch.uint8, device="cuda")
    k, v = memory[-n:].view(c["k_codes"].shape), memory[:n].view(c["k_codes"].shape)
    k.copy_(c["k_codes"])
    v.copy_(c["v_codes"])
    cache = kvq.Cache(k, v, c["k_scales"].cuda(), c["v_scales"].cuda(), 16)
    want = plain.attention(c, q, tables, lens, 1, SCALE, plain.window_rule(5, 1))
    for _ in range(20):
        assert_close(window(cache, q, tables, lens, 5, 1, 1), want, lens)


def test_small_calls_on_memory_that_changes():
    # caches of few pages and heads, new tensors each time: equal results twice, all finite
    g = torch.Generator().manual_seed(11)
    for i in range(150):
        H, G, R, n = (int(torch.randint(1, b, (1,), generator=g)) for b in (6, 5, 10, 4))
        lens = [int(torch.randint(0, 300, (1,), generator=g)) for _ in range(n)]
        c, tables = make(lens, H, 16, i)
        q = queries(n * R, H * G, i)
        cache = on_gpu(c)
        a = window(cache, q, tables, lens, 50, 3, R, most=max(max(lens), 1))
        b = tree(cache, q, random_mask(n, R, i), tables, lens, R, most=max(max(lens), 1))
        again = window(cache, q, tables, lens, 50, 3, R, most=max(max(lens), 1))
        assert torch.equal(a, again) and bool(torch.isfinite(a.float()).all() & torch.isfinite(b.float()).all())
