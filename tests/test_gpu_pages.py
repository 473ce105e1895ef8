"""The page pool, forks and the commit of an accepted path on the GPU: every table, count and
cache byte equal to plain Python's (oracle/masked.py)."""
import random

import pytest
import torch

import fp8_paged_kv_kvq_gb300 as kvq
import oracle.masked as plain

pytestmark = pytest.mark.gpu
PLANES = ("k_codes", "v_codes", "k_scales", "v_scales")


def cache_of(slots, H, bs, seed=0):
    g = torch.Generator().manual_seed(seed)
    codes = [torch.randint(0, 256, (slots, H, 128), generator=g, dtype=torch.uint8).cuda() for _ in range(2)]
    scales = [torch.rand(slots, H, generator=g).cuda() for _ in range(2)]
    return kvq.Cache(codes[0], codes[1], scales[0], scales[1], bs)


def planes(cache):
    return {n: getattr(cache, n).cpu().clone() for n in PLANES}


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def err_word():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


def pool_pair(pages, free=None):
    """A pool on the GPU and its plain twin; `free`: the stack from the bottom."""
    gpu, cpu = kvq.PagePool.empty(pages), plain.Pool(pages)
    if free is not None:
        cpu.free = list(free)
        cpu.refs = [0 if i in set(free) else 1 for i in range(pages)]
        gpu.free_pages[:len(free)] = ints(list(free))
        gpu.ref_counts.copy_(ints(cpu.refs))
        gpu.state[0] = len(free)
    return gpu, cpu


def assert_pool(gpu, cpu):
    torch.cuda.synchronize()
    assert gpu.state.tolist() == [len(cpu.free), 0, 0, 0]
    assert gpu.free_pages[:len(cpu.free)].tolist() == cpu.free
    assert gpu.ref_counts.tolist() == cpu.refs
    assert not bool(gpu.marks.any())


@pytest.mark.parametrize("n,width,pages", [(1, 1, 1), (1, 40, 64), (7, 9, 100), (300, 5, 2000), (2500, 3, 9000),
                                           (3, 3000, 9001)])
def test_alloc_and_free(n, width, pages):
    r = random.Random(n)
    order = list(range(pages))
    r.shuffle(order)
    gpu, cpu = pool_pair(pages, order)
    tables = [[-7] * width for _ in range(n)]
    t = ints(tables)
    begin = [r.randint(0, width) for _ in range(n)]
    end = [r.randint(b, width) for b in begin]
    err = err_word()
    kvq.pages_alloc(gpu, t, ints(begin), ints(end), err)
    cpu.alloc(tables, begin, end)
    assert t.tolist() == tables
    assert_pool(gpu, cpu)
    some = [r.randint(b, e) for b, e in zip(begin, end)]
    kvq.pages_free(gpu, t, ints(begin), ints(some), err)
    cpu.release(tables, begin, some)
    assert_pool(gpu, cpu)
    kvq.pages_free(gpu, t, ints(some), ints(end), err)
    cpu.release(tables, some, end)
    assert_pool(gpu, cpu)
    assert t.tolist() == tables and int(err) == 0 and sum(cpu.refs) == 0


def test_pool_runs_out():
    """The first request that does not fit and all that want pages after it get -1; what the pool
    has left stays."""
    for n in (5, 1500):
        need = [0] * n
        need[1], need[2], need[3] = 4, 7, 1
        need[n - 1] = 2
        gpu, cpu = pool_pair(10)
        tables = [[-3] * 8 for _ in range(n)]
        t, err = ints(tables), err_word()
        kvq.pages_alloc(gpu, t, ints([0] * n), ints(need), err)
        cpu.alloc(tables, [0] * n, need)
        assert t.tolist() == tables and tables[1][:4] == [9, 8, 7, 6] and tables[2][:7] == [-1] * 7
        assert_pool(gpu, cpu)
        assert int(err) == kvq.ERRF_NO_PAGES and len(cpu.free) == 6
    gpu, cpu = pool_pair(0 + 4, [])
    t, err = ints([[5, 5]]), err_word()
    kvq.pages_alloc(gpu, t, ints([0]), ints([2]), err)
    assert t.tolist() == [[-1, -1]] and int(err) == kvq.ERRF_NO_PAGES
    assert_pool(gpu, cpu)


def test_bad_ranges_and_entries():
    gpu, cpu = pool_pair(8)
    t, err = ints([[0, 1], [2, 3], [4, 5]]), err_word()
    kvq.pages_alloc(gpu, t, ints([-1, 2, 0]), ints([1, 1, 3]), err)
    assert t.tolist() == [[0, 1], [2, 3], [4, 5]] and int(err) == kvq.ERRF_CONTEXT_RANGE
    assert_pool(gpu, cpu)
    kvq.pages_alloc(gpu, t, ints([0, 0, 0]), ints([2, 1, 0]))
    err = err_word()
    kvq.pages_free(gpu, t, ints([-1, 2, 0]), ints([1, 1, 3]), err)
    assert int(err) == kvq.ERRF_CONTEXT_RANGE
    cpu.alloc([[0] * 2, [0] * 2], [0, 0], [2, 1])
    assert_pool(gpu, cpu)
    # a page twice, a page that nobody holds, no page, pages outside the pool
    held = t[0, 0].item()
    t2, err = ints([[held, held, 0, -1, 8, 2 ** 30, -2 ** 31]]), err_word()
    kvq.pages_free(gpu, t2, ints([0]), ints([7]), err)
    cpu.release([[held]], [0], [1])
    assert_pool(gpu, cpu)
    assert int(err) == kvq.ERRF_PAGE_STATE | kvq.ERRF_BLOCK_RANGE


def test_release_of_shared_pages_in_order():
    """Pages with several references, given back by many requests at once."""
    r = random.Random(5)
    pages, n, width = 70000, 64, 900
    gpu, cpu = pool_pair(pages, [])
    tables = [[r.randrange(pages) for _ in range(width)] for _ in range(n)]
    for x in range(pages):
        cpu.refs[x] = 0
    for row in tables:
        for x in row:
            cpu.refs[x] += 1
    for x in range(0, pages, 3):
        cpu.refs[x] += 1 if cpu.refs[x] else 0
    gpu.ref_counts.copy_(ints(cpu.refs))
    err = err_word()
    kvq.pages_free(gpu, ints(tables), ints([0] * n), ints([width] * n), err)
    cpu.release(tables, [0] * n, [width] * n)
    assert_pool(gpu, cpu)
    assert int(err) == 0 and len(cpu.free) > 10000


@pytest.mark.parametrize("bs", [1, 16, 64])
@pytest.mark.parametrize("H", [1, 3, 8])
@pytest.mark.parametrize("children", [1, 5, 300])
def test_fork(bs, H, children):
    r = random.Random(bs + H + children)
    np_, width, pages = 4, 6, 700
    gpu, cpu = pool_pair(pages)
    cache = cache_of(pages * bs, H, bs)
    lens = [0, width * bs, r.randint(1, width * bs), r.randint(1, width * bs)]
    tables = [[-1] * width for _ in range(np_)]
    cpu.alloc(tables, [0] * np_, [-(-x // bs) for x in lens])
    t = ints([[-1] * width for _ in range(np_)])
    kvq.pages_alloc(gpu, t, ints([0] * np_), ints([-(-x // bs) for x in lens]))
    parents = [r.choice([-1, 0, 1, 2, 3, 3]) for _ in range(children)]
    child = [[-9] * width for _ in range(children)]
    ct, cn, err = ints(child), ints([77] * children), err_word()
    want = planes(cache)
    kvq.pages_fork(cache, gpu, ints(parents), t, ints(lens), ct, cn, err)
    got_lens, copies = cpu.fork(parents, tables, lens, child, bs)
    assert cn.tolist() == got_lens and ct.tolist() == child
    assert_pool(gpu, cpu)
    for src, dst, n in copies:
        for x in want.values():
            x[dst:dst + n] = x[src:src + n]
    for name, x in planes(cache).items():
        assert torch.equal(x.view(torch.uint8), want[name].view(torch.uint8)), name
    assert int(err) == 0
    held = [-(-x // bs) for x in got_lens]
    kvq.pages_free(gpu, ct, ints([0] * children), ints(held), err)
    cpu.release(child, [0] * children, held)
    assert_pool(gpu, cpu)


def test_fork_without_pages_and_bad_parents():
    bs, width = 16, 3
    gpu, cpu = pool_pair(6)
    cache = cache_of(6 * bs, 2, bs)
    tables = [[-1] * width for _ in range(2)]
    cpu.alloc(tables, [0, 0], [2, 2])
    t = ints([[-1] * width for _ in range(2)])
    kvq.pages_alloc(gpu, t, ints([0, 0]), ints([2, 2]))
    parents, child = [0, 1, 0, 0, 1], [[-9] * width for _ in range(5)]
    ct, cn, err = ints(child), ints([1] * 5), err_word()
    kvq.pages_fork(cache, gpu, ints(parents), t, ints([20, 32]), ct, cn, err)
    lens, _ = cpu.fork(parents, tables, [20, 32], child, bs)
    assert cn.tolist() == lens == [20, 32, 20, 0, 32] and ct.tolist() == child
    assert int(err) == kvq.ERRF_NO_PAGES
    assert_pool(gpu, cpu)
    err = err_word()
    kvq.pages_fork(cache, gpu, ints([2, 10 ** 9]), t, ints([20, 32]), ct[:2], cn[:2], err)
    assert int(err) == kvq.ERRF_PATH_RANGE and cn[:2].tolist() == [0, 0]
    err = err_word()
    kvq.pages_fork(cache, gpu, ints([0, 1]), t, ints([-1, 49]), ct[:2], cn[:2], err)
    assert int(err) == kvq.ERRF_CONTEXT_RANGE and cn[:2].tolist() == [0, 0]
    assert_pool(gpu, cpu)
    # a parent's page outside the pool is passed on, not counted and not copied
    bad = t.clone()
    bad[1, 0] = 6
    bad[0, 1] = -4
    err = err_word()
    kvq.pages_free(gpu, ct[2:3], ints([1]), ints([2]))
    cpu.release([ct[2].tolist()], [1], [2])
    before = planes(cache)
    kvq.pages_fork(cache, gpu, ints([1, 0]), bad, ints([20, 32]), ct[:2], cn[:2], err)
    assert int(err) == kvq.ERRF_BLOCK_RANGE
    torch.cuda.synchronize()
    assert all(torch.equal(before[k], v) for k, v in planes(cache).items())


def commit_reference(want, tables, lens, paths, counts, R, bs):
    new = []
    for row, L, path, n in zip(tables, lens, paths, counts):
        moved = {name: x.clone() for name, x in want.items()}
        for a in range(n):
            f, t = L - R + path[a], L - R + a
            fs, ts = row[f // bs] * bs + f % bs, row[t // bs] * bs + t % bs
            for name, x in want.items():
                moved[name][ts] = x[fs]
        want.update(moved)
        new.append(L - R + n)
    return new


@pytest.mark.parametrize("H,bs", [(1, 16), (3, 16), (8, 64), (2, 1)])
@pytest.mark.parametrize("R", [1, 2, 7, 64, 300])
def test_commit(H, bs, R):
    """Random ascending paths, overlapping sources and places among them, page ends inside."""
    r = random.Random(R + H)
    n = 9
    lens = [R, R + 1] + [r.randint(R, R + 90) for _ in range(n - 2)]
    pages = [-(-x // bs) for x in lens]
    order = list(range(sum(pages)))
    r.shuffle(order)
    width = max(pages)
    tables = [[order.pop() for _ in range(p)] + [-1] * (width - p) for p in pages]
    paths = []
    for i in range(n):
        k = [0, R, r.randint(0, R)][min(i, 2)]
        paths.append(sorted(r.sample(range(R), k)))
    counts = [len(p) for p in paths]
    cache = cache_of(sum(pages) * bs, H, bs)
    want = planes(cache)
    new = commit_reference(want, tables, lens, paths, counts, R, bs)
    padded = ints([p + [-5] * (R - len(p)) for p in paths])
    err = err_word()
    cl = ints(lens)
    got = kvq.tree_commit(cache, padded, ints(counts), ints(tables), cl, err_flags=err)
    assert got.tolist() == new and cl.tolist() == lens and int(err) == 0
    for name, x in planes(cache).items():
        assert torch.equal(x.view(torch.uint8), want[name].view(torch.uint8)), name


def test_commit_in_place_idle_and_bad_paths():
    R, bs, H = 4, 16, 2
    lens = [20, 0, 30, 30, 30, 3, 40, 30]
    tables = [[2 * i, 2 * i + 1] for i in range(8)]
    paths = [[1, 3, 0, 0], [0] * 4, [2, 1, 0, 0], [0, 4, 0, 0], [1, 1, 0, 0], [0] * 4, [0] * 4, [-1, 0, 0, 0]]
    counts = [2, 0, 2, 2, 2, 1, 1, 1]
    cache = cache_of(16 * bs, H, bs)
    want = planes(cache)
    commit_reference(want, tables[:1], lens[:1], paths[:1], counts[:1], R, bs)
    cl, err = ints(lens), err_word()
    kvq.tree_commit(cache, ints(paths), ints(counts), ints(tables), cl, new_lens=cl, err_flags=err)
    assert cl.tolist() == [18, 0, 30, 30, 30, 3, 40, 30]
    assert int(err) == kvq.ERRF_PATH_RANGE | kvq.ERRF_CONTEXT_RANGE
    for name, x in planes(cache).items():
        assert torch.equal(x.view(torch.uint8), want[name].view(torch.uint8)), name
    # counts outside [0, R]
    err = err_word()
    got = kvq.tree_commit(cache, ints(paths[:2]), ints([5, -1]), ints(tables[:2]), ints([20, 0]), err_flags=err)
    assert got.tolist() == [20, 0] and int(err) == kvq.ERRF_PATH_RANGE | kvq.ERRF_CONTEXT_RANGE
    # pages outside the cache: those rows are not moved, the others are
    bad = [[0, 99]]
    err = err_word()
    want = planes(cache)
    got = kvq.tree_commit(cache, ints([[1, 2, 3, 0]]), ints([3]), ints(bad), ints([18]), err_flags=err)
    for name in PLANES:
        want[name][14] = want[name][15].clone()
    assert got.tolist() == [17] and int(err) == kvq.ERRF_BLOCK_RANGE
    for name, x in planes(cache).items():
        assert torch.equal(x.view(torch.uint8), want[name].view(torch.uint8)), name


def test_captured_calls():
    """alloc, fork, commit and free in one graph, replayed: the pool comes back to where it was."""
    bs, H, width = 16, 2, 4
    gpu, cpu = pool_pair(40)
    cache = cache_of(40 * bs, H, bs)
    t, lens = ints([[-1] * width]), ints([37])
    kvq.pages_alloc(gpu, t, ints([0]), ints([3]))
    ct, cn, new = ints([[-1] * width] * 3), ints([0] * 3), ints([0] * 3)
    parents, zero, three, four = ints([0, -1, 0]), ints([0] * 3), ints([3, 0, 3]), ints([4, 0, 4])
    paths, counts = ints([[1, 2], [0, 0], [0, 1]]), ints([1, 0, 2])
    err = err_word()

    def step():
        kvq.pages_fork(cache, gpu, parents, t, lens, ct, cn, err)
        kvq.pages_alloc(gpu, ct, three, four, err)
        kvq.tree_commit(cache, paths, counts, ct, cn, new, err)
        kvq.pages_free(gpu, ct, zero, four, err)

    step()
    torch.cuda.synchronize()
    before = [x.clone() for x in gpu.tensors()]
    first = ct.tolist(), new.tolist()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(5):
        g.replay()
    torch.cuda.synchronize()
    assert int(err) == 0 and (ct.tolist(), new.tolist()) == first and new.tolist() == [36, 0, 37]
    for a, b in zip(before, gpu.tensors()):
        assert torch.equal(a, b)
    # a freed page is copied over at most by its next holder: the parent's rows are its own still
    assert gpu.state[0].item() == 37


def test_a_serving_step():
    """The operators as they are used: two samples of a prompt, a tree drafted for each and verified,
    the accepted path committed, the pages behind it given back, then a windowed decode step with the
    pages outside the window given back as well."""
    torch.manual_seed(3)
    bs, H, Hq, R, L = 16, 2, 8, 6, 45
    gpu = kvq.PagePool.empty(64)
    cache = kvq.Cache.empty(64 * bs, H, 128, bs)
    width = 8
    err = err_word()
    t = ints([[-1] * width])
    kvq.pages_alloc(gpu, t, ints([0]), ints([3]), err)
    j = torch.arange(L, device="cuda")
    rows = lambda n: torch.randn(n, H, 128, device="cuda").to(torch.bfloat16)
    slots = lambda table, pos: table[pos // bs].long() * bs + pos % bs
    kvq.quantize_scatter(cache, rows(L), rows(L), slots(t[0], j), err)
    ct, cl = ints([[-1] * width] * 2), ints([0, 0])
    kvq.pages_fork(cache, gpu, ints([0, 0]), t, ints([L]), ct, cl, err)
    kvq.pages_free(gpu, t, ints([0]), ints([3]), err)
    # drafted tokens stored behind the context
    grown = cl + R
    kvq.pages_alloc(gpu, ct, ints([3, 3]), (grown + bs - 1) // bs, err)
    for r in range(2):
        kvq.quantize_scatter(cache, rows(R), rows(R), slots(ct[r], L + torch.arange(R, device="cuda")), err)
    mask = torch.tensor([[1], [2], [0b101], [0b1010], [0b10101], [0b101010]], dtype=torch.int32, device="cuda")
    mask = mask[None].repeat(2, 1, 1).contiguous()
    q = torch.randn(2 * R, Hq, 128, device="cuda").to(torch.bfloat16)

    def reference(q, tables, lens, R, rule):
        c = dict(block_size=bs, **planes(cache))
        return plain.attention(c, q.cpu(), tables.cpu(), lens, R, 0.09, rule)[0]

    out = kvq.paged_decode_tree(cache, q, mask, ct, grown, 64, 0.09, R, err_flags=err)
    ref = reference(q, ct, [L + R] * 2, R, plain.tree_rule(mask.cpu()))
    assert float((out.cpu().double() - ref).abs().max()) < 2e-2
    before = planes(cache)
    pages = ct.cpu().tolist()
    lens = kvq.tree_commit(cache, ints([[0, 2, 4, 0, 0, 0], [1, 3, 5, 0, 0, 0]]), ints([3, 2]), ct, grown,
                           err_flags=err)
    assert lens.tolist() == [L + 3, L + 2]
    after = planes(cache)
    for r, path in enumerate(([0, 2, 4], [1, 3])):
        for a, node in enumerate(path):
            to, fro = L + a, L + node
            for n in PLANES:
                assert torch.equal(after[n][pages[r][to // bs] * bs + to % bs],
                                   before[n][pages[r][fro // bs] * bs + fro % bs])
    kvq.pages_free(gpu, ct, (lens + bs - 1) // bs, (grown + bs - 1) // bs, err)
    # a windowed step over what is left; pages between sink and window are given back before
    q1 = torch.randn(2, Hq, 128, device="cuda").to(torch.bfloat16)
    ref = reference(q1, ct, lens.tolist(), 1, plain.window_rule(12, 4))
    kvq.pages_free(gpu, ct, ints([1, 1]), ints([2, 2]), err)
    ct[:, 1] = -1
    out = kvq.paged_decode_window(cache, q1, ct, lens, 64, 12, 0.09, num_sinks=4, err_flags=err)
    assert float((out.cpu().double() - ref).abs().max()) < 2e-2
    kvq.pages_free(gpu, ct, ints([0, 0]), (lens + bs - 1) // bs, err)
    torch.cuda.synchronize()
    assert int(err) == 0 and gpu.state[0].item() == 64 and not bool(gpu.ref_counts.any())
