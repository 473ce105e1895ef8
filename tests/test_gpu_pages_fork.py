"""Forks of parents whose block tables hold entries that are no pages of the pool."""
import pytest
import torch

import fp8_paged_kv_kvq_gb300 as kvq
from test_gpu_pages import cache_of, err_word, ints, planes, pool_pair

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [40, -4, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("bs", [1, 16])
def test_a_parents_page_outside_the_pool_is_passed_on(bad, bs):
    """As it is, neither counted nor copied, also as a partly filled last page: no page is taken for it,
    and the children behind it get the pages that they would get without it."""
    pages, width, H = 40, 4, 2
    gpu, _ = pool_pair(pages)
    cache = cache_of(pages * bs, H, bs)
    t = ints([[-1] * width for _ in range(3)])
    kvq.pages_alloc(gpu, t, ints([0] * 3), ints([4, 4, 3]))            # pages 39 .. 29
    part = bs // 2                                                     # (pages of one token: none is partly filled)
    lens = [2 * bs + part, 3 * bs + part, bs + part]
    t[0, 2], t[1, 1] = bad, bad
    refs, free = gpu.ref_counts.clone(), int(gpu.state[0])
    ct, cn, err = ints([[-9] * width for _ in range(5)]), ints([7] * 5), err_word()
    before, table = planes(cache), t.tolist()
    kvq.pages_fork(cache, gpu, ints([2, 0, 1, 0, 2]), t, ints(lens), ct, cn, err)
    last = (lambda k: [28 - k]) if part else (lambda k: [-9])
    passed = [bad] if part else [-9]
    want = [table[2][:1] + last(0) + [-9] * 2,
            table[0][:2] + passed + [-9],
            [table[1][0], bad, table[1][2]] + last(1),
            table[0][:2] + passed + [-9],
            table[2][:1] + last(2) + [-9] * 2]
    assert ct.tolist() == want and cn.tolist() == [lens[2], lens[0], lens[1], lens[0], lens[2]]
    assert int(err) == kvq.ERRF_BLOCK_RANGE
    shared = [table[2][0]] * 2 + table[0][:2] * 2 + [table[1][0], table[1][2]]
    for page in shared + ([28, 27, 26] if part else []):
        refs[page] += 1
    assert gpu.ref_counts.tolist() == refs.tolist()
    assert gpu.state.tolist() == [free - (3 if part else 0), 0, 0, 0]
    copies = [(table[2][1], 28), (table[1][3], 27), (table[2][1], 26)] if part else []
    for src, dst in copies:
        for x in before.values():
            x[dst * bs:dst * bs + part] = x[src * bs:src * bs + part]
    for name, x in planes(cache).items():
        assert torch.equal(x.view(torch.uint8), before[name].view(torch.uint8)), name


def test_no_page_is_wanted_for_a_page_outside_the_pool():
    """Of an empty pool such a child is a child, the others are none."""
    bs, width = 16, 2
    gpu, _ = pool_pair(4)
    cache = cache_of(4 * bs, 1, bs)
    t = ints([[-1] * width for _ in range(2)])
    kvq.pages_alloc(gpu, t, ints([0, 0]), ints([2, 2]))
    t[1, 1] = 4
    ct, cn, err = ints([[-9] * width for _ in range(3)]), ints([7] * 3), err_word()
    kvq.pages_fork(cache, gpu, ints([0, 1, 0]), t, ints([20, 20]), ct, cn, err)
    assert cn.tolist() == [0, 20, 0] and ct.tolist() == [[-9, -9], [int(t[1, 0]), 4], [-9, -9]]
    assert int(err) == kvq.ERRF_NO_PAGES | kvq.ERRF_BLOCK_RANGE
    assert gpu.state.tolist() == [0, 0, 0, 0]
    refs = [1] * 4
    refs[int(t[1, 0])] = 2
    assert gpu.ref_counts.tolist() == refs
