"""Windowed and tree attention over the paged cache, the commit of an accepted path, and forked pages.

Operators of a serving step over the FP8 paged cache (e4m3 codes, one fp32 scale per (token, KV head) row):

  window  attention of each request's last R tokens over a sliding window of its cached tokens
          and the first few, which stay visible (sinks)
  tree    attention of a tree of R drafted tokens, the last R cached ones of each request, over the
          context before them and over their ancestors
  commit  the rows of the accepted drafted tokens moved together behind the context
  fork    children that continue their parents' sequences: whole pages shared, the last partly
          filled one copied, pages for the tokens to come, and all of them given back

With ``own`` False, ``run`` computes them with elementary torch operations in fp32, rounded once
at the end; with ``own`` True it calls this library.
"""
import math
import random

import torch

own = False

D = 128


def listed():
    return [
        # One request far into its text, one new token, the pages between sinks and window given back:
        # the smallest call, where latency counts.
        dict(name="window_one", op="window", n=1, idle=0, r=1, hq=32, h=8, lo=100000, hi=100000, window=1024,
             sinks=4, block=16, evicted=True),
        # A decode step of 64 requests, three of them idle, most of them longer than the window.
        dict(name="window_decode_64", op="window", n=64, idle=3, r=1, hq=32, h=8, lo=500, hi=32768, window=4096,
             sinks=4, block=16, evicted=False),
        # A verify step of 4 rows, 64 query heads, an odd window, pages of 64 tokens.
        dict(name="window_verify_37x4", op="window", n=37, idle=0, r=4, hq=64, h=8, lo=100, hi=20000, window=1001,
             sinks=1, block=64, evicted=True),
        # Chunks of 2,048 prompt tokens at the end of contexts of up to 16,384.
        dict(name="window_chunks_4x2048", op="window", n=4, idle=0, r=2048, hq=32, h=8, lo=9000, hi=16384, window=4096,
             sinks=16, block=64, evicted=False),
        # One request with a small tree of 16 drafted tokens.
        dict(name="tree_one_16", op="tree", n=1, idle=0, r=16, hq=32, h=8, lo=2000, hi=2000, block=16),
        # Five requests, trees of 25 nodes, 7 query heads per KV head.
        dict(name="tree_5x25", op="tree", n=5, idle=0, r=25, hq=28, h=4, lo=2500, hi=9001, block=32),
        # A full batch with trees of 8 nodes, two requests idle.
        dict(name="tree_batch_128x8", op="tree", n=128, idle=2, r=8, hq=32, h=8, lo=1000, hi=8192, block=16),
        # Wide trees of 64 nodes and 64 query heads: 512 rows per KV head.
        dict(name="tree_wide_8x64", op="tree", n=8, idle=0, r=64, hq=64, h=8, lo=4096, hi=16384, block=64),
        # What follows a single request's verify step.
        dict(name="commit_one_16", op="commit", n=1, r=16, h=8, lo=2000, hi=2000, most=6, block=16),
        # What follows a batch's verify step over wide trees.
        dict(name="commit_512x64", op="commit", n=512, r=64, h=8, lo=200, hi=2000, most=16, block=64),
        # Eight samples of one prompt.
        dict(name="fork_1_to_8", op="fork", parents=1, children=8, h=8, lo=1003, hi=1003, grow=16, block=16),
        # Four beams for each of 64 requests, pages of 64 tokens.
        dict(name="fork_64_to_256", op="fork", parents=64, children=256, h=8, lo=100, hi=4000, grow=64, block=64),
    ]


#: What a drawn attention case costs at most, in products of a query row with a key row, and its cache rows.
_PAIRS = 4 * 32 * 2048 * 4096
_ROWS = 5_000_000


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["window", "window", "window", "tree", "tree", "tree", "commit", "fork"])
    h = rng.choice([1, 2, 3, 4, 8, 8])
    block = rng.choice([16, 16, 32, 64, 128])
    if op == "commit":
        r = _log_uniform(rng, 2, 96)
        hi = _log_uniform(rng, r, 2000)
        return dict(op=op, n=_log_uniform(rng, 1, 512), r=r, h=h, lo=rng.randint(r, hi), hi=hi,
                    most=rng.randint(1, min(r, 16)), block=block)
    if op == "fork":
        children = _log_uniform(rng, 1, 256)
        hi = _log_uniform(rng, 1, 4000)
        return dict(op=op, parents=rng.randint(1, min(children, 64)), children=children, h=h, lo=rng.randint(1, hi), hi=hi,
                    grow=_log_uniform(rng, 1, 300), block=block)
    hq = h * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    n = _log_uniform(rng, 1, 128)
    idle = rng.choice([0, 0, rng.randint(0, n - 1)])
    if op == "tree":
        r = _log_uniform(rng, 1, 96)
        most = min(16384, _PAIRS // (n * hq * r), _ROWS // (n * h))
        hi = _log_uniform(rng, r, max(r, most))
        return dict(op=op, n=n, idle=idle, r=r, hq=hq, h=h, lo=rng.randint(r, hi), hi=hi, block=block)
    r = rng.choice([1, 1, rng.randint(2, 8), _log_uniform(rng, 9, 2048)])
    window = _log_uniform(rng, 1, 8192)
    sinks = rng.choice([0, 1, 4, 4, rng.randint(5, 200)])
    evicted = rng.random() < 0.5
    # (with the pages in between given back, only sinks and window take cache rows)
    most = 200000 if evicted and n * h * (window + sinks + r + 3 * block) < _ROWS else min(65536, _ROWS // (n * h))
    while n > 1 and n * hq * r * min(most, window + sinks) > _PAIRS:
        n //= 2
        idle = 0
    hi = _log_uniform(rng, r, max(r, most))
    return dict(op=op, n=n, idle=idle, r=r, hq=hq, h=h, lo=rng.randint(r, hi), hi=hi, window=window, sinks=sinks,
                block=block, evicted=evicted)


def _lens(case):
    """The requests' cached tokens, the longest of them the case's bound; idle requests of a padded batch have none."""
    n, lo, hi = case.get("n", case.get("parents")), case["lo"], case["hi"]
    r = random.Random("%d %d %d" % (n, lo, hi))
    lens = [_log_uniform(r, lo, hi) for _ in range(n)]
    at = r.randrange(n)
    for i in r.sample(range(n), case.get("idle", 0)):
        lens[i] = 0
    lens[at] = hi
    return lens


def _cache(slots, h, g):
    """Codes and scales of a cache of N(0, 1) rows, in the library's row format."""
    codes = [torch.empty(slots, h, D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.empty(slots, h, device="cuda") for _ in range(2)]
    step = max(1, 2 ** 24 // (h * D))
    for c, s in zip(codes, scales):
        for i in range(0, slots, step):
            x = torch.randn(min(step, slots - i), h, D, generator=g, device="cuda")
            scale = x.abs().amax(dim=-1) / 448
            c[i:i + step] = (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            s[i:i + step] = scale
    return dict(k_codes=codes[0], v_codes=codes[1], k_scales=scales[0], v_scales=scales[1])


def _tables(keep, width, spare, c):
    """Block tables int32 [n, width] with pages of their own, in random order, for the entries listed in `keep`
    (the others -1), and the number of pages."""
    total = sum(len(k) for k in keep)
    order = torch.randperm(total + spare, generator=c)[:total].to(torch.int32)
    tables = torch.full((len(keep), width), -1, dtype=torch.int32)
    at = 0
    for row, k in zip(tables, keep):
        row[torch.tensor(k, dtype=torch.int64)] = order[at:at + len(k)]
        at += len(k)
    return tables, total + spare


def _tree_mask(n, r, c):
    """A random tree for each request: node i hangs on an earlier node or on the context; bit j of row i is set
    where node j is node i itself or one of its ancestors.  int32 words [n, r, ceil(r / 32)]."""
    seen = torch.zeros(n, r, r, dtype=torch.bool)
    for i in range(r):
        parent = torch.where(torch.rand(n, generator=c) < 0.15, torch.full((n,), -1),
                             (torch.rand(n, generator=c) * i).long().clamp(max=i - 1))
        if i:
            seen[:, i] = seen[torch.arange(n), parent.clamp(min=0)] & (parent >= 0)[:, None]
        seen[:, i, i] = True
    words = torch.zeros(n, r, (r + 31) // 32 * 32, dtype=torch.int64)
    words[..., :r] = seen
    words = (words.view(n, r, -1, 32) << torch.arange(32)).sum(dim=-1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32)


def _accepted(case, c):
    """The accepted path of each request: ascending nodes of its tree (whose first level is as wide as the path is
    long, so that a path's rows move to places that hold none of them and a pass can be repeated)."""
    n, r = case["n"], case["r"]
    paths = torch.zeros(n, r, dtype=torch.int32)
    lens = torch.randint(0, case["most"] + 1, (n,), generator=c)
    for i, m in enumerate(lens.tolist()):
        first = int(torch.randint(0, 2, (1,), generator=c)) if 0 < m < r else m
        m = min(m, r - m + first) if m < r else m
        first = min(first, m)
        lens[i] = m
        rest = torch.randperm(max(r - m, 0), generator=c)[:m - first].sort().values + m
        paths[i, :m] = torch.cat([torch.arange(first), rest]).to(torch.int32)
    return paths, lens.to(torch.int32)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    c = torch.Generator().manual_seed(int(seed))
    op, h, bs = case["op"], case["h"], case["block"]
    lens = _lens(case)
    pages = [-(-n // bs) for n in lens]
    width = max(pages) + 1
    if op == "fork":
        children = case["children"]
        width += -(-case["grow"] // bs) + 1
        tables, total = _tables([list(range(p)) for p in pages], width, 0, c)
        # the pages in use first, then those of the pool: enough for every child, and some more
        total_free = children * (2 + case["grow"] // bs) + 7
        parents = torch.randint(0, case["parents"], (children,), generator=c).to(torch.int32)
        lens_t = torch.tensor(lens, dtype=torch.int32)
        child = lens_t[parents.long()]
        used = torch.zeros(total + total_free, dtype=torch.int32)
        used[:total] = 1
        free = torch.zeros(total + total_free, dtype=torch.int32)
        free[:total_free] = torch.arange(total, total + total_free)
        return dict(case=case, **_cache((total + total_free) * bs, h, g), tables=tables.cuda(), lens=lens_t.cuda(),
                    parents=parents.cuda(), child_tables=torch.full((children, width), -1, dtype=torch.int32, device="cuda"),
                    child_lens=torch.zeros(children, dtype=torch.int32, device="cuda"), ref=used.cuda(), free=free.cuda(),
                    state=torch.tensor([total_free, 0, 0, 0], dtype=torch.int32, device="cuda"),
                    marks=torch.zeros((total + total_free + 31) // 32, dtype=torch.int32, device="cuda"),
                    none=torch.zeros(children, dtype=torch.int32, device="cuda"), held=((child + bs - 1) // bs).cuda(),
                    grown=((child + case["grow"] + bs - 1) // bs).cuda())
    keep = [list(range(p)) for p in pages]
    if op == "window" and case["evicted"]:
        # pages that neither the sinks nor any row's window reach have gone back to the pool
        keep = []
        for n in lens:
            first = max(0, n - case["r"] + 1 - case["window"])
            keep.append([p for p in range(-(-n // bs)) if p * bs < case["sinks"] or p * bs + bs > first])
    tables, total = _tables(keep, width, 5, c)
    s = dict(case=case, **_cache(total * bs, h, g), tables=tables.cuda(),
             lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    if op == "commit":
        paths, counts = _accepted(case, c)
        s.update(paths=paths.cuda(), counts=counts.cuda(), new_lens=torch.zeros(case["n"], dtype=torch.int32, device="cuda"))
        return s
    n, r, hq = case["n"], case["r"], case["hq"]
    s.update(q=(1.5 * torch.randn(n * r, hq, D, generator=g, device="cuda")).to(torch.bfloat16),
             out=torch.zeros(n * r, hq, D, dtype=torch.bfloat16, device="cuda"), most=max(lens), scale=1 / math.sqrt(D))
    if op == "tree":
        s["mask"] = _tree_mask(n, r, c).cuda()
    if own:
        import fp8_paged_kv_kvq_gb300 as kvq
        if op == "tree":
            size = kvq.paged_decode_tree_workspace_size(n, r, hq, h, D, bs, s["most"])
        else:
            size = kvq.paged_decode_window_workspace_size(n, r, hq, h, D, bs, s["most"], case["window"], case["sinks"])
        s["workspace"] = torch.empty(max(size, 1), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# The plain forms.


def _plain_attention(s, a, b, pos, seen):
    """Requests a .. b - 1: their rows over the cached tokens at pos [b - a, keys], of which row i sees
    seen[:, i] [b - a, R, keys]; rows that see none are zero."""
    case = s["case"]
    n, r, hq, h, bs = b - a, case["r"], case["hq"], case["h"], case["block"]
    page = s["tables"][a:b].gather(1, (pos // bs).clamp(0, s["tables"].shape[1] - 1)).long()
    any_row = seen.any(dim=1)
    slot = torch.where(any_row, page * bs + pos % bs, torch.zeros_like(pos))
    f8 = torch.float8_e4m3fn
    q = s["q"][a * r:b * r].view(n, r, h, hq // h, D).float().permute(0, 2, 3, 1, 4).reshape(n * h, -1, D)
    k = (s["k_codes"].view(f8)[slot].float() * s["k_scales"][slot][..., None]).permute(0, 2, 3, 1).reshape(n * h, D, -1)
    score = torch.bmm(q, k).mul_(s["scale"])
    del k
    score.view(n, h, hq // h, r, -1).masked_fill_(~seen[:, None, None], -math.inf)
    top = score.amax(dim=-1, keepdim=True)
    score.sub_(torch.where(top > -math.inf, top, torch.zeros_like(top))).exp_()
    v = (s["v_codes"].view(f8)[slot].float() * s["v_scales"][slot][..., None]).permute(0, 2, 1, 3).reshape(n * h, -1, D)
    total = score.sum(dim=-1, keepdim=True)
    o = torch.bmm(score, v).div_(torch.where(total > 0, total, torch.ones_like(total)))
    o = o.view(n, h, hq // h, r, D).permute(0, 3, 1, 2, 4).reshape(n * r, hq, D)
    s["out"][a * r:b * r] = o.to(torch.bfloat16)


def _groups(case, keys):
    """Requests in groups whose gathered keys and scores stay at a few GB."""
    cost = keys * max(case["h"] * D, case["hq"] * case["r"])
    size = max(1, int(2 ** 29 // max(cost, 1)))
    return [(a, min(case["n"], a + size)) for a in range(0, case["n"], size)]


def _plain_window(s):
    case = s["case"]
    r, window, sinks, most = case["r"], case["window"], case["sinks"], s["most"]
    wide = min(most, window + r - 1)                    # tokens that some row's window reaches
    few = min(sinks, most)
    dev = s["q"].device
    for a, b in _groups(case, wide + few):
        length = s["lens"][a:b].long()[:, None]
        first = (length - wide).clamp(min=0)
        pos = torch.cat([torch.arange(few, device=dev).expand(b - a, few), first + torch.arange(wide, device=dev)], dim=1)
        # a sink that the window's tokens hold as well counts there
        there = torch.cat([pos[:, :few] < first, torch.ones(b - a, wide, dtype=torch.bool, device=dev)], dim=1)
        row = (length - r + torch.arange(r, device=dev))[..., None]          # the rows' own positions
        p = pos[:, None]
        _plain_attention(s, a, b, pos, there[:, None] & (p <= row) & ((p < sinks) | (p > row - window)))


def _plain_tree(s):
    case, mask = s["case"], s["mask"]
    r = case["r"]
    dev = s["q"].device
    for a, b in _groups(case, s["most"]):
        length = s["lens"][a:b].long()
        pos = torch.arange(s["most"], device=dev).expand(b - a, -1)
        node = pos - (length - r)[:, None]                                   # < 0: context
        at = node.clamp(0, r - 1)
        word = mask[a:b].gather(2, (at // 32)[:, None].expand(-1, r, -1))
        bit = (word >> (at % 32)[:, None].int()) & 1
        seen = (node < 0)[:, None] | ((bit != 0) & (node < r)[:, None])
        _plain_attention(s, a, b, pos, seen)


_PLANES = ("k_codes", "v_codes", "k_scales", "v_scales")


def _plain_commit(s):
    case = s["case"]
    r, bs = case["r"], case["block"]
    base = s["lens"].long()[:, None] - r
    take = torch.arange(r, device=base.device) < s["counts"][:, None]
    src, dst = (base + s["paths"])[take], (base + torch.arange(r, device=base.device))[take]
    of = take.nonzero()[:, 0]
    src = s["tables"][of, src // bs].long() * bs + src % bs
    dst = s["tables"][of, dst // bs].long() * bs + dst % bs
    for name in _PLANES:
        s[name][dst] = s[name][src]
    s["new_lens"].copy_(s["lens"] - r + s["counts"])


def _plain_take(s, need):
    """Pages for a list of requests that need as many each (int64): rows of the pool's top, in order."""
    state = s["state"]
    last = need.cumsum(0)
    at = state[0].long() - 1 - torch.arange(int(last[-1]), device=need.device)
    got = s["free"][at]
    s["ref"][got.long()] = 1
    state[0] -= last[-1].int()
    return got


def _plain_fork(s):
    case = s["case"]
    bs = case["block"]
    tables, out = s["tables"][s["parents"].long()], s["child_tables"]
    s["child_lens"].copy_(s["lens"][s["parents"].long()])
    length = s["child_lens"].long()
    full, rest = length // bs, length % bs
    col = torch.arange(out.shape[1], device=out.device)
    shared = col < full[:, None]
    out.copy_(torch.where(shared, tables, out))
    s["ref"].index_add_(0, tables[shared].long(), torch.ones_like(tables[shared]))
    part = (rest > 0).nonzero()[:, 0]
    got = _plain_take(s, (rest > 0).long())
    out[part, full[part]] = got
    tok = torch.arange(bs, device=out.device)
    live = tok < rest[part][:, None]
    src = (tables[part, full[part]].long()[:, None] * bs + tok)[live]
    dst = (got.long()[:, None] * bs + tok)[live]
    for name in _PLANES:
        s[name][dst] = s[name][src]
    # pages for the tokens to come
    new = (col >= s["held"][:, None]) & (col < s["grown"][:, None])
    out[new] = _plain_take(s, new.sum(dim=1))
    # and the children's pages given back: those that nobody holds any more, by their numbers
    freed = out[col < s["grown"][:, None]]
    s["ref"].index_add_(0, freed.long(), torch.full_like(freed, -1))
    held = torch.zeros(s["ref"].shape[0], dtype=torch.bool, device=out.device)
    held[freed.long()] = True
    back = (held & (s["ref"] == 0)).nonzero()[:, 0].int()
    n = int(s["state"][0])
    s["free"][n:n + back.numel()] = back
    s["state"][0] += back.numel()


def run(state):
    s = state
    case = s["case"]
    op = case["op"]
    if own:
        import fp8_paged_kv_kvq_gb300 as kvq
        cache = kvq.Cache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"], case["block"])
        if op == "window":
            kvq.paged_decode_window(cache, s["q"], s["tables"], s["lens"], s["most"], case["window"], s["scale"],
                                    num_sinks=case["sinks"], rows_per_request=case["r"], out=s["out"],
                                    workspace=s.get("workspace"))
        elif op == "tree":
            kvq.paged_decode_tree(cache, s["q"], s["mask"], s["tables"], s["lens"], s["most"], s["scale"],
                                  rows_per_request=case["r"], out=s["out"], workspace=s.get("workspace"))
        elif op == "commit":
            kvq.tree_commit(cache, s["paths"], s["counts"], s["tables"], s["lens"], new_lens=s["new_lens"])
        else:
            pool = kvq.PagePool(s["ref"], s["free"], s["state"], s["marks"])
            kvq.pages_fork(cache, pool, s["parents"], s["tables"], s["lens"], s["child_tables"], s["child_lens"])
            kvq.pages_alloc(pool, s["child_tables"], s["held"], s["grown"])
            kvq.pages_free(pool, s["child_tables"], s["none"], s["grown"])
    else:
        dict(window=_plain_window, tree=_plain_tree, commit=_plain_commit, fork=_plain_fork)[op](s)
    if op in ("window", "tree"):
        return s["out"]
    f8 = torch.float8_e4m3fn
    got = dict(k_codes=s["k_codes"].view(f8), v_codes=s["v_codes"].view(f8), k_scales=s["k_scales"],
               v_scales=s["v_scales"])
    if op == "commit":
        got["new_lens"] = s["new_lens"]
    else:
        got.update(child_tables=s["child_tables"], child_lens=s["child_lens"], ref=s["ref"],
                   free=s["free"], num_free=s["state"][:1])
    return got


def work(case):
    h, bs = case["h"], case["block"]
    lens = _lens(case)
    row = h * 2 * (D + 4)                               # a cached token
    if case["op"] == "commit":
        c = torch.Generator().manual_seed(0)
        moved = int(_accepted(case, c)[1].sum())
        return dict(bytes=2 * moved * row + 4 * moved + 12 * case["n"], flops=0)
    if case["op"] == "fork":
        # the children's parents are drawn with the inputs: their mean
        each = case["children"] / case["parents"]
        copied = sum(n % bs for n in lens) * each
        pages = sum(-(-(n + case["grow"]) // bs) for n in lens) * each
        return dict(bytes=int(2 * copied * row + 20 * pages), flops=0)
    r, hq = case["r"], case["hq"]
    moved = case["n"] * r * hq * D * 4                  # queries and outputs
    pairs = 0
    for n in lens:
        if n == 0:
            continue
        if case["op"] == "tree":
            # (some 8 nodes of a random tree see each other)
            moved += n * row + r * ((r + 31) // 32) * 4 + 4 * -(-n // bs)
            pairs += r * (n - r) + r * min(r, 8)
            continue
        first = max(0, n - r + 1 - case["window"])
        tokens = n - first + min(case["sinks"], first)
        moved += tokens * row + 4 * -(-tokens // bs)
        for p in range(n - r, n):
            low = max(0, p + 1 - case["window"])
            pairs += p + 1 - low + min(case["sinks"], low)
    return dict(bytes=moved, flops=4 * D * hq * pairs)


# ---------------------------------------------------------------------------
# The definitions in 64 bits.


def _exact_attention(s):
    case = s["case"]
    r, h, bs = case["r"], case["h"], case["block"]
    out = torch.zeros_like(s["out"], dtype=torch.float64)
    rows = out.view(case["n"], r, h, -1, D)
    queries = s["q"].view(case["n"], r, h, -1, D)
    f8 = torch.float8_e4m3fn
    for i, length in enumerate(s["lens"].tolist()):
        if length == 0:
            continue
        i0 = length - r
        if case["op"] == "tree":
            first, few = 0, 0
        else:
            first = max(0, i0 + 1 - case["window"])
            few = min(case["sinks"], first)
        tokens = torch.cat([torch.arange(few), torch.arange(first, length)]).to(s["q"].device)
        slot = s["tables"][i, tokens // bs].long() * bs + tokens % bs
        own_pos = torch.arange(i0, length, device=tokens.device)
        if case["op"] == "tree":
            words = s["mask"][i].long() & 0xFFFFFFFF
            bits = ((words[:, :, None] >> torch.arange(32, device=words.device)) & 1).flatten(1)[:, :r].bool()
            hidden = torch.cat([torch.zeros(r, i0, dtype=torch.bool, device=words.device), ~bits], dim=1)
        else:
            far = own_pos[:, None] - tokens[None, :]
            hidden = (far < 0) | ((far >= case["window"]) & (tokens >= case["sinks"])[None, :])
        for head in range(h):
            k = s["k_codes"][slot, head].view(f8).double() * s["k_scales"][slot, head].double()[:, None]
            v = s["v_codes"][slot, head].view(f8).double() * s["v_scales"][slot, head].double()[:, None]
            for a in range(0, r, 256):
                q = queries[i, a:a + 256, head].double()
                x = torch.einsum("igd,kd->igk", q, k) * s["scale"]
                w = torch.softmax(x.masked_fill(hidden[a:a + 256, None], -math.inf), dim=-1)
                rows[i, a:a + 256, head] = torch.einsum("igk,kd->igd", w, v)
    return out


def _values(s):
    f8 = torch.float8_e4m3fn
    return dict(k_codes=s["k_codes"].view(f8).double(), v_codes=s["v_codes"].view(f8).double(),
                k_scales=s["k_scales"].double(), v_scales=s["v_scales"].double())


def _exact_commit(s):
    bs, r = s["case"]["block"], s["case"]["r"]
    tables, lens = s["tables"].tolist(), s["lens"].tolist()
    dst, src, new = [], [], []
    for t, length, path, count in zip(tables, lens, s["paths"].tolist(), s["counts"].tolist()):
        for to, node in enumerate(path[:count]):
            a, b = length - r + node, length - r + to
            src.append(t[a // bs] * bs + a % bs)
            dst.append(t[b // bs] * bs + b % bs)
        new.append(length - r + count)
    got = _values(s)
    for x in got.values():
        x[dst] = x[src]
    got["new_lens"] = torch.tensor(new, dtype=torch.int32, device=s["lens"].device)
    return got


def _exact_fork(s):
    case = s["case"]
    bs = case["block"]
    tables, lens = s["tables"].tolist(), s["lens"].tolist()
    child = s["child_tables"].tolist()
    ref, free, n = s["ref"].tolist(), s["free"].tolist(), int(s["state"][0])
    got = _values(s)
    src, dst = [], []

    def take():
        nonlocal n
        n -= 1
        ref[free[n]] += 1
        return free[n]

    for row, parent in zip(child, s["parents"].tolist()):
        for j in range(lens[parent] // bs):
            row[j] = tables[parent][j]
            ref[row[j]] += 1
        left = lens[parent] % bs
        if left:
            j = lens[parent] // bs
            row[j] = take()
            src += [tables[parent][j] * bs + t for t in range(left)]
            dst += [row[j] * bs + t for t in range(left)]
    for x in got.values():
        x[dst] = x[src]
    length = [lens[p] for p in s["parents"].tolist()]
    for row, have in zip(child, length):
        for j in range(-(-have // bs), -(-(have + case["grow"]) // bs)):
            row[j] = take()
    back = set()
    for row, have in zip(child, length):
        for page in row[:-(-(have + case["grow"]) // bs)]:
            ref[page] -= 1
            if ref[page] == 0:
                back.add(page)
    for page in sorted(back):
        free[n] = page
        n += 1
    dev = s["lens"].device
    as_int = lambda x: torch.tensor(x, dtype=torch.int32, device=dev)
    got.update(child_tables=as_int(child), child_lens=as_int(length), ref=as_int(ref), free=as_int(free),
               num_free=as_int([n]))
    return got


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "commit":
        return _exact_commit(s)
    if case["op"] == "fork":
        return _exact_fork(s)
    return _exact_attention(s)
