"""Refusals of the windowed and tree attention, the commit and the page pool: every call
here is answered on the host, before anything could be launched."""
import ctypes

import pytest
import torch

import fp8_paged_kv_kvq_gb300 as kvq
from fp8_paged_kv_kvq_gb300 import build as kbuild

OK, INVALID, UNSUPPORTED, MISALIGNED, WS_SMALL = 0, 1, 2, 3, 4
P = ctypes.c_void_p
NULL = dict(q=0, bt=0, cl=0, out=0, ws=0, mask=0)


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kvq.load()


def _cache(head_dim=128, ptr=0x10000, H=8, bs=16, slots=640):
    return kvq._CacheStruct(ptr, ptr + 0x100000, ptr + 0x200000, ptr + 0x300000, slots, H, head_dim, bs)


CALL = dict(q=0x1000, mask=0x2000, N=3, R=4, hq=32, bt=0x3000, mb=8, cl=0x4000, most=100, window=64,
            sinks=4, scale=0.1, out=0x5000, ws=0x6000, size=1 << 40, err=0)


def _window(lib, cache=None, **changes):
    a = dict(CALL, **changes)
    c = cache if cache is not None else _cache()
    return lib.kvq_paged_decode_window(
        ctypes.byref(c), P(a["q"]), a["N"], a["R"], a["hq"], P(a["bt"]), a["mb"], P(a["cl"]),
        a["most"], a["window"], a["sinks"], a["scale"], P(a["out"]), P(a["ws"]), a["size"],
        P(a["err"]), P(0))


def _tree(lib, cache=None, **changes):
    a = dict(CALL, **changes)
    c = cache if cache is not None else _cache()
    return lib.kvq_paged_decode_tree(
        ctypes.byref(c), P(a["q"]), P(a["mask"]), a["N"], a["R"], a["hq"], P(a["bt"]), a["mb"],
        P(a["cl"]), a["most"], a["scale"], P(a["out"]), P(a["ws"]), a["size"], P(a["err"]), P(0))


@pytest.mark.parametrize("changes,status", [
    (dict(N=0), OK), (dict(N=0, **{k: 0 for k in ("q", "bt", "cl", "out", "ws")}), OK),
    (dict(N=-1), INVALID), (dict(R=0), INVALID), (dict(hq=0), INVALID), (dict(hq=30), INVALID),
    (dict(mb=-1), INVALID), (dict(most=-1), INVALID), (dict(q=0), INVALID), (dict(bt=0), INVALID),
    (dict(cl=0), INVALID), (dict(out=0), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(R=2049), UNSUPPORTED), (dict(N=65536), UNSUPPORTED),
    (dict(N=65535, most=1 << 30), UNSUPPORTED), (dict(q=0x1008), MISALIGNED),
    (dict(out=0x5008), MISALIGNED), (dict(bt=0x3002), MISALIGNED), (dict(cl=0x4002), MISALIGNED),
    (dict(ws=0x6008), MISALIGNED), (dict(err=2), MISALIGNED),
])
@pytest.mark.parametrize("call", [_window, _tree])
def test_attention_refusals(lib, call, changes, status):
    assert call(lib, **changes) == status


@pytest.mark.parametrize("call", [_window, _tree])
def test_attention_refuses_more_than_31_bits_number(lib, call):
    # chunks of 32 tokens of four heads (R G <= 32), 1,024 requests a launch
    assert call(lib, cache=_cache(H=1), N=1024, R=1, hq=1, most=1 << 26) == UNSUPPORTED
    assert call(lib, cache=_cache(H=4), N=2048, R=1, hq=4, most=1 << 26) == UNSUPPORTED
    assert call(lib, N=1, R=4, most=(1 << 30) + 1) == UNSUPPORTED
    assert call(lib, N=1, R=4, most=(1 << 31) - 1) == UNSUPPORTED


@pytest.mark.parametrize("changes,status", [
    (dict(window=0), INVALID), (dict(window=-5), INVALID), (dict(sinks=-1), INVALID)])
def test_window_refusals(lib, changes, status):
    assert _window(lib, **changes) == status


@pytest.mark.parametrize("changes,status", [
    (dict(mask=0), INVALID), (dict(mask=0x2002), MISALIGNED), (dict(R=1025, hq=8), UNSUPPORTED)])
def test_tree_refusals(lib, changes, status):
    assert _tree(lib, **changes) == status


@pytest.mark.parametrize("call", [_window, _tree])
def test_attention_cache_refusals(lib, call):
    assert call(lib, cache=_cache(head_dim=64)) == UNSUPPORTED
    assert call(lib, cache=_cache(bs=8)) == UNSUPPORTED
    assert call(lib, cache=_cache(bs=24)) == UNSUPPORTED
    assert call(lib, cache=_cache(bs=0)) == INVALID
    assert call(lib, cache=_cache(ptr=0x10008)) == MISALIGNED
    assert call(lib, cache=_cache(slots=1 << 31)) == UNSUPPORTED


def test_workspace_sizes(lib):
    w, t = kvq.paged_decode_window_workspace_size, kvq.paged_decode_tree_workspace_size
    for n, r in ((1, 1), (64, 1), (3, 4), (2, 300)):
        assert w(n, r, 32, 8, 128, 16, 4096, 1000, 4) == t(n, r, 32, 8, 128, 16, 4096)
        assert t(n + 1, r, 32, 8, 128, 16, 4096) >= t(n, r, 32, 8, 128, 16, 4096)
    for bad in (dict(window=0), dict(num_sinks=-1)):
        assert w(**{**dict(num_requests=1, rows_per_request=1, num_q_heads=8, num_kv_heads=8,
                           head_dim=128, block_size=16, max_context_len=100, window=9), **bad}) == 0
    assert t(1, 1025, 8, 8, 128, 16, 2000) == 0 and t(1, 1, 9, 8, 128, 16, 2000) == 0
    size = t(3, 4, 32, 8, 128, 16, 100)
    if size:
        assert _tree(lib, size=size - 1) == WS_SMALL and _window(lib, ws=0) == WS_SMALL


COMMIT = dict(acc=0x1000, lens=0x2000, N=3, R=8, bt=0x3000, mb=8, cl=0x4000, new=0x5000, err=0)


def _commit(lib, cache=None, **changes):
    a = dict(COMMIT, **changes)
    c = cache if cache is not None else _cache()
    return lib.kvq_tree_commit(ctypes.byref(c), P(a["acc"]), P(a["lens"]), a["N"], a["R"],
                               P(a["bt"]), a["mb"], P(a["cl"]), P(a["new"]), P(a["err"]), P(0))


@pytest.mark.parametrize("changes,status", [
    (dict(N=0), OK), (dict(N=0, acc=0, lens=0, bt=0, cl=0, new=0), OK), (dict(N=-1), INVALID),
    (dict(R=0), INVALID), (dict(mb=-1), INVALID), (dict(R=1025), UNSUPPORTED), (dict(acc=0), INVALID),
    (dict(lens=0), INVALID), (dict(bt=0), INVALID), (dict(cl=0), INVALID), (dict(new=0), INVALID),
    (dict(acc=0x1002), MISALIGNED), (dict(lens=0x2001), MISALIGNED), (dict(bt=0x3002), MISALIGNED),
    (dict(cl=0x4002), MISALIGNED), (dict(new=0x5002), MISALIGNED), (dict(err=1), MISALIGNED),
])
def test_commit_refusals(lib, changes, status):
    assert _commit(lib, **changes) == status
    assert _commit(lib, cache=_cache(head_dim=64)) == UNSUPPORTED


def _pool(pages=40, refs=0x1000, free=0x2000, state=0x3000, marks=0x4000):
    return kvq._PagePoolStruct(refs, free, state, marks, pages)


RANGES = dict(bt=0x5000, N=3, mb=8, begin=0x6000, end=0x7000, err=0)


@pytest.mark.parametrize("changes,status", [
    (dict(N=0), OK), (dict(N=-1), INVALID), (dict(mb=-1), INVALID), (dict(bt=0), INVALID),
    (dict(begin=0), INVALID), (dict(end=0), INVALID), (dict(mb=(1 << 20) + 1), UNSUPPORTED),
    (dict(bt=0x5002), MISALIGNED), (dict(begin=0x6001), MISALIGNED), (dict(end=0x7002), MISALIGNED),
    (dict(err=2), MISALIGNED),
    (dict(pool=dict(pages=-1)), INVALID), (dict(pool=dict(refs=0)), INVALID),
    (dict(pool=dict(free=0)), INVALID), (dict(pool=dict(state=0)), INVALID),
    (dict(pool=dict(marks=0)), INVALID), (dict(pool=dict(state=0x3002)), MISALIGNED),
])
def test_page_range_refusals(lib, changes, status):
    a = dict(RANGES, **changes)
    pool = _pool(**a.get("pool", {}))
    for fn in (lib.kvq_pages_alloc, lib.kvq_pages_free):
        assert fn(ctypes.byref(pool), P(a["bt"]), a["N"], a["mb"], P(a["begin"]), P(a["end"]),
                  P(a["err"]), P(0)) == status


FORK = dict(parents=0x8000, M=4, bt=0x9000, N=2, mb=8, cl=0xA000, ct=0xB000, cn=0xC000, err=0)


@pytest.mark.parametrize("changes,status", [
    (dict(M=0), OK), (dict(M=-1), INVALID), (dict(N=-1), INVALID), (dict(mb=-1), INVALID),
    (dict(M=4097), UNSUPPORTED), (dict(mb=(1 << 20) + 1), UNSUPPORTED), (dict(parents=0), INVALID),
    (dict(bt=0), INVALID), (dict(cl=0), INVALID), (dict(ct=0), INVALID), (dict(cn=0), INVALID),
    (dict(ct=0x9000), INVALID), (dict(cn=0xA000), INVALID), (dict(ct=0xB002), MISALIGNED),
    (dict(parents=0x8002), MISALIGNED), (dict(cn=0xC002), MISALIGNED), (dict(err=2), MISALIGNED),
    (dict(pages=41), INVALID),                      # more pages than the cache has
])
def test_fork_refusals(lib, changes, status):
    a = dict(FORK, **changes)
    c, pool = _cache(), _pool(pages=a.get("pages", 40))
    assert lib.kvq_pages_fork(ctypes.byref(c), ctypes.byref(pool), P(a["parents"]), a["M"],
                              P(a["bt"]), a["N"], a["mb"], P(a["cl"]), P(a["ct"]), P(a["cn"]),
                              P(a["err"]), P(0)) == status


def test_bindings_reject_bad_tensors():
    """dtypes, shapes, layouts and devices are checked before the library is called."""
    cache = kvq.Cache.empty(64, 2, 128, 16, device="cpu")
    q = torch.zeros(6, 8, 128, dtype=torch.bfloat16)
    bt, cl = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    mask = torch.zeros(2, 3, 1, dtype=torch.int32)
    good = dict(q=q, block_tables=bt, context_lens=cl, max_context_len=64, sm_scale=0.1,
                rows_per_request=3)
    for bad in (dict(q=q.float()), dict(q=q[:, :, :64]), dict(q=q[:5]), dict(q=q[0]),
                dict(q=q.transpose(0, 1)), dict(block_tables=bt.long()), dict(block_tables=bt[0]),
                dict(block_tables=bt.T), dict(context_lens=cl.long()), dict(context_lens=cl[:1]),
                dict(rows_per_request=2), dict(rows_per_request=0), dict(out=q[:3]),
                dict(out=q.float()), dict(err_flags=torch.zeros(1)),
                dict(workspace=torch.zeros(8, 8, dtype=torch.uint8).T)):
        with pytest.raises(ValueError):
            kvq.paged_decode_window(cache, window=8, **{**good, **bad})
        with pytest.raises(ValueError):
            kvq.paged_decode_tree(cache, tree_mask=mask, **{**good, **bad})
    for bad in (mask.long(), mask[:1], torch.zeros(2, 3, 2, dtype=torch.int32)):
        with pytest.raises(ValueError):
            kvq.paged_decode_tree(cache, tree_mask=bad, **good)
    with pytest.raises(ValueError, match="current CUDA device"):
        kvq.paged_decode_window(cache, window=8, **good)            # host tensors
    with pytest.raises(ValueError, match="current CUDA device"):
        kvq.paged_decode_tree(cache, tree_mask=mask, **good)

    acc = torch.zeros(2, 3, dtype=torch.int32)
    good = dict(accepted=acc, accepted_lens=cl, block_tables=bt, context_lens=cl)
    for bad in (dict(accepted=acc.long()), dict(accepted=acc[:1]), dict(accepted=acc[0]),
                dict(accepted_lens=cl[:1]), dict(block_tables=bt.T), dict(context_lens=cl.long()),
                dict(new_lens=cl.long()), dict(err_flags=torch.zeros(1))):
        with pytest.raises(ValueError):
            kvq.tree_commit(cache, **{**good, **bad})
    with pytest.raises(ValueError, match="current CUDA device"):
        kvq.tree_commit(cache, **good)

    pool = kvq.PagePool.empty(4, device="cpu")
    assert pool.state.tolist() == [4, 0, 0, 0] and pool.free_pages.tolist() == [0, 1, 2, 3]
    for fn in (kvq.pages_alloc, kvq.pages_free):
        for args in ((bt.long(), cl, cl), (bt[0], cl, cl), (bt, cl[:1], cl), (bt, cl, cl.long())):
            with pytest.raises(ValueError):
                fn(pool, *args)
        bad_pool = kvq.PagePool(pool.ref_counts, pool.free_pages[:3], pool.state, pool.marks)
        with pytest.raises(ValueError):
            fn(bad_pool, bt, cl, cl)
        with pytest.raises(ValueError, match="current CUDA device"):
            fn(pool, bt, cl, cl)
    ct, cn, parents = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), \
        torch.zeros(3, dtype=torch.int32)
    good = dict(parents=parents, block_tables=bt, context_lens=cl, child_tables=ct, child_lens=cn)
    for bad in (dict(parents=parents.long()), dict(parents=parents[:2]), dict(block_tables=bt[:, :3]),
                dict(context_lens=cn), dict(child_tables=ct.long()), dict(child_lens=cl),
                dict(err_flags=torch.zeros(1))):
        with pytest.raises(ValueError):
            kvq.pages_fork(cache, pool, **{**good, **bad})
    with pytest.raises(ValueError, match="current CUDA device"):
        kvq.pages_fork(cache, pool, **good)
