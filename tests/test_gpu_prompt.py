"""kvq_prompt_attention on the GPU against dense fp64 attention (oracle/prompt.py).

Tolerance.  Of an output o = sum_j w_j v_j the kernel rounds: the output to
bf16 (2^-8 |o|); every probability to bf16 for the product (2^-8 sum_j w_j |v_j|,
the sum's denominator is not rounded); the score of 128 binary32 additions and
its scaling, an absolute error of at most 130 2^-23 max_j sm_scale sum_d |q_d k_jd|
=: e (one unit in the last place per addition, as the tensor cores may truncate),
which moves numerator and denominator by a relative e each; the exponentials,
2^-20 each; and the two sums of up to L terms, a unit in the last place per
addition, L 2^-22 together.  In all
    |err| <= 2^-8 |o| + (2^-8 + 2 e + 2^-19 + L 2^-22) sum_j w_j |v_j|."""
import numpy as np
import pytest
import torch

import fp8_paged_kv_kvq_gb300 as kvq
import oracle
import oracle.prompt as plain
import workloads
from kvq_testlib import assert_attention_close

pytestmark = pytest.mark.gpu
SCALE = 128 ** -0.5


def _inputs(T, hq, H, seed, spread=1.5):
    """q, k, v [T, heads, 128] as views of one fused projection output on the GPU."""
    g = workloads.generator(seed, 301)
    qkv = torch.randn(T, (hq + 2 * H) * 128, generator=g)
    qkv[:, :hq * 128] *= spread
    qkv = qkv.to(torch.bfloat16).cuda()
    return (qkv[:, :hq * 128].view(T, hq, 128), qkv[:, hq * 128:(hq + H) * 128].view(T, H, 128),
            qkv[:, (hq + H) * 128:].view(T, H, 128))


def _cu(lens, first=0):
    return torch.tensor([first] + list(first + np.cumsum(lens)), dtype=torch.int32, device="cuda")


def bound(ref, mag, dot, lens):
    e = 130 * 2.0 ** -23 * dot
    return 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * e + 2.0 ** -19 + max(lens) * 2.0 ** -22) * mag


def assert_close(got, q, k, v, lens, scale=SCALE):
    """Rows of the packed sequences (inputs already cut to them)."""
    ref, mag, dot = plain.prompt_attention(q, k, v, lens, scale)
    tol = bound(ref, mag, dot, lens)
    err = (got.cpu().double() - ref).abs()
    assert bool(torch.isfinite(got).all())
    worst = float((err / tol.clamp(min=1e-300)).max()) if err.numel() else 0.0
    print(f"worst |err| / bound {worst:.3f}")
    assert worst <= 1.0


def _run(lens, hq, H, seed, scale=SCALE, tail=0, first=0, spread=1.5, most=None):
    T = first + int(sum(lens)) + tail
    q, k, v = _inputs(T, hq, H, seed, spread)
    out = torch.full((T, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.prompt_attention(q, k, v, _cu(lens, first), max(lens) if most is None else most, scale,
                         out=out, err_flags=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    end = T - tail
    assert torch.all(out[:first] == 7) and torch.all(out[end:] == 7)
    assert_close(out[first:end], q[first:end], k[first:end], v[first:end], lens, scale)


@pytest.mark.parametrize("lens", [
    [1], [2], [63], [64], [65], [127], [128], [129], [255, 256, 257], [1, 1, 1, 1, 1],
    [0, 5, 0, 0, 130, 0], [31, 32, 33, 383], [512, 1, 640], [1000],
])
@pytest.mark.parametrize("hq,H", [(32, 8), (3, 3), (7, 1)])
def test_lengths(lens, hq, H):
    _run(lens, hq, H, seed=sum(lens) + hq)


@pytest.mark.parametrize("hq,H", [(1, 1), (2, 1), (6, 2), (10, 2), (12, 2), (14, 2), (16, 2), (9, 1),
                                  (32, 2), (64, 1), (127, 1), (128, 1)])
def test_head_groups(hq, H):
    _run([200, 77, 300], hq, H, seed=hq)


@pytest.mark.parametrize("lens,hq,H", [([640], 4, 1), ([1290], 4, 1), ([129, 500], 6, 2),
                                       ([128, 256, 384], 4, 2), ([2500], 2, 1), ([257], 128, 1)])
def test_split_keys(lens, hq, H):
    """So few units that two chains share a row tile, each over every other key tile (one, two, an
    odd and an even number of them)."""
    _run(lens, hq, H, seed=sum(lens))


@pytest.mark.parametrize("lens,hq,H", [([650], 32, 8), ([2000], 16, 2), ([1500, 1500], 8, 2),
                                       ([3700], 8, 1), ([2900, 1], 8, 1)])
def test_split_keys_of_more_units_than_sms(lens, hq, H):
    """Split keys where some SMs take a second unit (and where the last of two sequences is one
    row, whose second chain has no key)."""
    _run(lens, hq, H, seed=sum(lens) + 1)


@pytest.mark.parametrize("hq,H", [(8, 2), (2, 2), (14, 2)])
def test_mixed_lengths(hq, H):
    """Tails, heads and whole short prompts side by side, among empty ones."""
    g = workloads.generator(31, hq)
    lens = []
    for _ in range(20):
        lens += torch.randint(0, 9, (4,), generator=g).tolist()
        lens += torch.randint(20, 200, (1,), generator=g).tolist()
    lens[7] = 700
    _run(lens, hq, H, seed=31, tail=5, first=3)


@pytest.mark.parametrize("lens,hq,H", [([700], 4, 1), ([1999], 8, 1), ([700, 300], 64, 16),
                                       ([2000, 1, 129], 28, 4), ([517], 128, 1)])
def test_each_key_counts_once(lens, hq, H):
    """Equal scores (queries of zeros) and values that are 1 in dim d at one key of the sequence and
    0 elsewhere: row i has 1 / (i + 1) there once it sees the key, and exactly 0 before.  A key
    dropped or counted twice at a tile's seam, or a row that sees one too many, cannot hide: the
    probabilities are all the same, so all that is left is the output's rounding (2^-8, and a few
    2^-23 of the sum and its reciprocal)."""
    q, k, v = _inputs(sum(lens), hq, H, seed=33)
    q.zero_()
    v.zero_()
    seams = [x + d for x in range(0, max(lens) + 128, 128) for d in (-1, 0, 1)]
    seams += list(range(31, max(lens), 32))[:30] + [x - 1 for x in lens] + [x - 2 for x in lens]
    g = workloads.generator(33, sum(lens))
    dims = torch.randperm(128, generator=g).tolist()
    a, want = 0, torch.zeros(sum(lens), 128, dtype=torch.float64)
    for L in lens:
        keys = sorted({x for x in seams if 0 <= x < L})[:128]
        for key, d in zip(keys, dims):
            v[a + key, :, d] = 1.0
            want[a + key:a + L, d] = 1.0 / torch.arange(key + 1, L + 1, dtype=torch.float64)
        a += L
    out = kvq.prompt_attention(q, k, v, _cu(lens), max(lens), SCALE)
    torch.cuda.synchronize()
    want = want[:, None, :].expand(-1, hq, -1)
    got = out.cpu().double()
    assert torch.equal(got == 0, want == 0)
    assert bool(((got - want).abs() <= (2.0 ** -8 + 2.0 ** -20) * want).all())


def test_longer_prompt():
    _run([2333, 130], 8, 2, seed=4)


@pytest.mark.parametrize("lens,hq,H", [([2900, 1500, 40, 700], 32, 8), ([1999, 1999], 28, 4),
                                       ([130] * 150, 16, 4)])
def test_many_units_per_cta(lens, hq, H):
    """Several times more units of work than the GPU has SMs, of very different lengths."""
    _run(lens, hq, H, seed=5)


@pytest.mark.parametrize("n", [32, 33, 600, 1500, 2048, 2049, 3000])
def test_many_sequences(n):
    """Many sequences, empty ones among them: counted by a warp, by all threads in one or several
    rounds, and so many that a unit is found over cu_seqlens itself."""
    g = workloads.generator(6, n)
    lens = torch.randint(0, 12, (n,), generator=g).tolist()
    lens[n // 2] = 300
    _run(lens, 4, 2, seed=6, tail=3, first=2)
    # one of them out of bounds: flagged
    T = int(sum(lens))
    q, k, v = _inputs(T, 4, 2, seed=6)
    cu = _cu(lens)
    cu[n // 2 + 1] = T + 1
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.prompt_attention(q, k, v, cu, 300, SCALE, err_flags=err)
    torch.cuda.synchronize()
    assert int(err.item()) == kvq.ERRF_SEQUENCE_RANGE


def test_rows_outside_the_sequences_stay():
    _run([70, 0, 200], 16, 4, seed=7, tail=150, first=33)
    _run([0, 0], 16, 4, seed=7, tail=9, most=0)


@pytest.mark.parametrize("hq,H", [(8, 2), (64, 16)])
@pytest.mark.parametrize("scale,spread", [(SCALE, 12.0), (1.0, 1.0), (1e-6, 1.0)])
def test_score_ranges(scale, spread, hq, H):
    """Peaked rows (one probability near 1), and rows of nearly equal scores."""
    _run([400, 150], hq, H, seed=9, scale=scale, spread=spread)


@pytest.mark.parametrize("hq,H", [(8, 2), (64, 32)])
def test_climbing_and_falling_scores(hq, H):
    """Scores that rise (fall) by many powers of two along the keys, so that running maxima move
    again and again (or never)."""
    L = 700
    q, k, v = _inputs(L, hq, H, seed=11)
    q.copy_(torch.ones_like(q))
    step = (torch.arange(L, device="cuda") / 3.0)[:, None, None]
    for sign in (1.0, -1.0):
        noise = torch.randn(L, H, 128, generator=workloads.generator(12, 1)).cuda()
        k.copy_((sign * step / 128 / SCALE + 0.05 * noise).to(torch.bfloat16))
        out = kvq.prompt_attention(q, k, v, _cu([L]), L, SCALE)
        torch.cuda.synchronize()
        assert_close(out, q, k, v, [L])


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("hq,H", [(8, 2), (2, 2), (64, 16)])
def test_unseen_infinities_and_nans_do_not_reach_a_row(bad, hq, H):
    """Keys and values of later tokens, of the next sequence and of the padding are infinite or
    NaN: rows before them are exact, rows that see an infinite value get it."""
    lens, tail = [150, 300, 37], 20
    T = sum(lens) + tail
    q, k, v = _inputs(T, hq, H, seed=13)
    clean_q, clean_k, clean_v = q.clone(), k.clone(), v.clone()
    spots = [100, 149, 150 + 130, 150 + 299, 486]       # tokens, one or two of each sequence
    v[spots, :, 3] = bad
    k[spots, :, 64] = bad
    q[spots] = 0                                       # (their own scores are NaN all the same)
    k[487:], v[487:], q[487:] = bad, bad, bad
    out = kvq.prompt_attention(q, k, v, _cu(lens), 300, SCALE)
    torch.cuda.synchronize()
    ref, mag, dot = plain.prompt_attention(clean_q, clean_k, clean_v, lens + [0], SCALE)
    tol = bound(ref, mag, dot, lens)
    clean = torch.zeros(T, dtype=torch.bool)
    clean[:100] = clean[150:280] = clean[450:486] = True
    err = (out.cpu().double() - ref).abs()
    assert bool(torch.isfinite(out[clean.cuda()]).all())
    assert bool((err <= tol)[clean].all())


@pytest.mark.parametrize("hq,H", [(8, 2), (64, 16)])
def test_seen_infinite_values(hq, H):
    """Infinite and NaN values with finite keys: rows that see one have it in that dim (infinities
    of both signs: NaN), every other element is the finite sum."""
    lens = [333, 70]
    T = sum(lens)
    q, k, v = _inputs(T, hq, H, seed=14)
    clean = v.clone()
    inf, nan = float("inf"), float("nan")
    for tok, dim, x in ((10, 5, inf), (140, 6, -inf), (300, 5, -inf), (200, 7, nan), (332, 8, inf),
                        (333, 9, nan), (400, 5, inf)):
        v[tok, :, dim] = x
        clean[tok, :, dim] = 0.0
    out = kvq.prompt_attention(q, k, v, _cu(lens), 333, SCALE)
    torch.cuda.synchronize()
    ref, mag, dot = plain.prompt_attention(q, k, clean, lens, SCALE)
    tol = bound(ref, mag, dot, lens)
    want = ref.clone()
    for tok, dim, x in ((10, 5, inf), (140, 6, -inf), (300, 5, -inf), (200, 7, nan), (332, 8, inf),
                        (333, 9, nan), (400, 5, inf)):
        want[tok:(333 if tok < 333 else T), :, dim] += x
    got = out.cpu().double()
    fin = torch.isfinite(want)
    assert bool((((got - want).abs() <= tol) | ~fin).all())
    assert bool((got[~fin].isnan() == want[~fin].isnan()).all())
    both = ~fin & ~want.isnan()
    assert bool((got[both] == want[both]).all())


@pytest.mark.parametrize("L,hq,H", [(400, 8, 2), (400, 64, 16)])
def test_seen_infinite_values_of_no_probability(L, hq, H):
    """An infinite value whose probability underflows: a row that sees it has that infinity or NaN
    (0 times it), never a finite value; every other element is the finite sum."""
    q, k, v = _inputs(L, hq, H, seed=34)
    q.fill_(1.0)
    k.mul_(1 / 64)
    spots = ((5, 3, float("inf")), (150, 4, float("-inf")), (390, 6, float("inf")))
    clean = v.clone()
    for tok, dim, x in spots:
        k[tok] = -30.0                                  # a score some 490 powers of two below
        v[tok, :, dim] = x
        clean[tok, :, dim] = 0.0
    out = kvq.prompt_attention(q, k, v, _cu([L]), L, SCALE)
    torch.cuda.synchronize()
    ref, mag, dot = plain.prompt_attention(q, k, clean, [L], SCALE)
    seen = torch.zeros(L, hq, 128, dtype=torch.bool)
    for tok, dim, x in spots:
        seen[tok:, :, dim] = True
    got = out.cpu().double()
    assert bool(((got - ref).abs() <= bound(ref, mag, dot, [L]))[~seen].all())
    for tok, dim, x in spots:
        y = got[tok:, :, dim]
        assert bool((y.isnan() | (y == x)).all())


@pytest.mark.parametrize("cu,most", [
    ([0, 50, 40, 100], 64),           # decreasing
    ([0, 30, 60, 101], 64),           # past the buffer
    ([-5, 30, 60, 100], 64),          # in front of it
    ([0, 30, 100, 100], 64),          # longer than max_seqlen
    ([0, 2_000_000_000, -2_000_000_000, 100], 2_000_000_000),
    ([0, 30, 60, 100], 0),
])
def test_bad_bounds_are_flagged_and_stay_in_the_buffers(cu, most):
    """Every access is checked against the buffers (shown by the kernel's own bounds checks); rows
    of other tensors around them stay as they were."""
    T, hq, H = 100, 8, 2
    q, k, v = _inputs(T, hq, H, seed=15)
    guard = torch.full((T + 400, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out = guard[200:200 + T]
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    kvq.prompt_attention(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), most, SCALE,
                         out=out, err_flags=err)
    torch.cuda.synchronize()
    assert int(err.item()) == kvq.ERRF_SEQUENCE_RANGE
    assert torch.all(guard[:200] == 7) and torch.all(guard[200 + T:] == 7)


def test_offsets_past_32_bits():
    """A token buffer of more than 2^31 elements, the sequences at its end."""
    hq, H, T = 32, 8, 360_000
    qkv = torch.zeros(T, (hq + 2 * H) * 128, dtype=torch.bfloat16, device="cuda")
    lens = [130, 300]
    first = T - sum(lens)
    g = workloads.generator(16, 1)
    qkv[first:] = torch.randn(sum(lens), qkv.shape[1], generator=g).to(torch.bfloat16).cuda()
    q = qkv[:, :hq * 128].view(T, hq, 128)
    k = qkv[:, hq * 128:(hq + H) * 128].view(T, H, 128)
    v = qkv[:, (hq + H) * 128:].view(T, H, 128)
    out = torch.zeros(T, hq, 128, dtype=torch.bfloat16, device="cuda")
    kvq.prompt_attention(q, k, v, _cu(lens, first), 300, SCALE, out=out)
    torch.cuda.synchronize()
    assert_close(out[first:], q[first:], k[first:], v[first:], lens)


def test_captured_replayed_and_on_another_stream():
    """A captured call replayed on new rows and other lengths below its bound; two streams at once."""
    hq, H, T = 16, 4, 600
    q, k, v = _inputs(T, hq, H, seed=17)
    cu = _cu([100, 400])
    out = torch.zeros(T, hq, 128, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kvq.prompt_attention(q, k, v, cu, 500, SCALE, out=out)
    for seed, lens in ((18, [500, 100]), (19, [3, 0]), (20, [255, 257])):
        for x, y in zip((q, k, v), _inputs(T, hq, H, seed)):
            x.copy_(y)
        cu.copy_(_cu(lens))
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        n = sum(lens)
        assert torch.all(out[n:] == 7)
        assert_close(out[:n], q[:n], k[:n], v[:n], lens)
    other = torch.zeros_like(out)
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    kvq.prompt_attention(q, k, v, cu, 500, SCALE, out=other, stream=side)
    kvq.prompt_attention(q, k, v, cu, 500, SCALE, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, other)                      # the same call gives the same bits
    assert_close(out[:512], q[:512], k[:512], v[:512], [255, 257])


@pytest.mark.parametrize("hq,H", [(4, 1), (64, 16)])
def test_strides_and_alignment_of_their_own(hq, H):
    """q, k, v and out with four different token strides, none a multiple of 32 bytes, each 16 bytes
    off a 32-byte boundary; what lies between the rows of out stays."""
    lens = [130, 9, 261]
    T = sum(lens)
    views = []
    for x, gap in zip(_inputs(T, hq, H, seed=26), (8, 24, 40)):
        heads = x.shape[1]
        buf = torch.full((T * (heads * 128 + gap) + 8,), 3.0, dtype=torch.bfloat16, device="cuda")
        views.append(buf.as_strided((T, heads, 128), (heads * 128 + gap, 128, 1), 8))
        views[-1].copy_(x)
    buf = torch.full((T, hq * 128 + 56), 7.0, dtype=torch.bfloat16, device="cuda")
    out = buf.as_strided((T, hq, 128), (hq * 128 + 56, 128, 1), 8)
    kvq.prompt_attention(*views, _cu(lens), 300, SCALE, out=out)
    torch.cuda.synchronize()
    assert torch.all(buf[:, :8] == 7) and torch.all(buf[:, hq * 128 + 8:] == 7)
    assert_close(out, *views, lens)


@pytest.mark.parametrize("hq,H", [(4, 1), (64, 16)])
def test_large_values(hq, H):
    """Values around 2^100, whose sums the unnormalised probabilities (below 2^16) may not push out
    of binary32: 2^100 2^16 350 < 2^125."""
    lens = [350, 40]
    q, k, v = _inputs(390, hq, H, seed=27, spread=8.0)
    v = (v.double() * 2.0 ** 97).clamp(-2.0 ** 100, 2.0 ** 100).to(torch.bfloat16)
    out = kvq.prompt_attention(q, k, v, _cu(lens), 350, SCALE)
    torch.cuda.synchronize()
    assert_close(out, q, k, v, lens)


@pytest.mark.parametrize("hq,H", [(4, 1), (64, 16)])
def test_values_near_the_top_of_the_range(hq, H):
    """Values of up to 2^119 under references that trail the rows' maxima by 2^15: the sums stay
    below sum_j p_j |v_j| with p_j <= 1, 2^119 350 < 2^128."""
    lens = [350, 40]
    q, k, v = _inputs(390, hq, H, seed=29)
    q.fill_(1.0)
    k.mul_(1 / 64)
    k[:128] += 15 / (128 * SCALE * float(np.log2(np.e)))     # the first sequence's oldest keys
    v = (v.double().abs().clamp(0.25, 4.0) * 2.0 ** 117).to(torch.bfloat16)
    out = kvq.prompt_attention(q, k, v, _cu(lens), 350, SCALE)
    torch.cuda.synchronize()
    assert_close(out, q, k, v, lens)


@pytest.mark.parametrize("hq,H", [(4, 1), (64, 16)])
@pytest.mark.parametrize("exponent", [-80, -110])
def test_small_values(exponent, hq, H):
    """Values around 2^-80 and 2^-110, under probabilities of 2^-16 for the reference's own score:
    products of 2^-126 and less are subnormal, each off by at most 2^-149, 350 2^-149 2^16 of the
    output in all, far below 2^-8 2^-110."""
    lens = [350, 40]
    q, k, v = _inputs(390, hq, H, seed=30)
    v = (v.double() * 2.0 ** exponent).to(torch.bfloat16)
    out = kvq.prompt_attention(q, k, v, _cu(lens), 350, SCALE)
    torch.cuda.synchronize()
    assert_close(out, q, k, v, lens)


@pytest.mark.parametrize("tail", [1, 2000, 15000])
def test_padding_does_not_change_the_sequences_rows(tail):
    """A sequence with padding behind it has the bits that it has alone: how its work is cut up
    goes by the sequences' bounds, not by the buffer's length."""
    L, hq, H = 900, 32, 8
    q, k, v = _inputs(L + tail, hq, H, seed=32)
    alone = kvq.prompt_attention(q[:L], k[:L], v[:L], _cu([L]), L, SCALE)
    out = kvq.prompt_attention(q, k, v, _cu([L]), L, SCALE)
    torch.cuda.synchronize()
    assert torch.equal(out[:L], alone)


def test_calls_that_follow_one_another():
    """Calls in a row that read what the last one wrote (rotated in place and stored, attended over,
    the outputs the next queries), of few units and of many, give the bits that they give with a
    wait after each."""
    def steps(wait):
        got = []
        for lens, hq, H in (([200, 90], 8, 2), ([300, 300, 41], 64, 16)):
            T = sum(lens)
            q, k, v = (x.clone() for x in _inputs(T, hq, H, seed=28))
            pos = torch.arange(T).cuda()
            cu, table = _cu(lens), plain.rope_table(T, 128).cuda()
            cache = kvq.Cache.empty(T, H)
            torch.cuda.synchronize()
            for _ in range(4):
                kvq.rope_quantize_scatter(cache, q, k, v, pos, table, pos, q_out=q, k_out=k)
                if wait:
                    torch.cuda.synchronize()
                q = kvq.prompt_attention(q, k, v, cu, 300, SCALE)
                if wait:
                    torch.cuda.synchronize()
            torch.cuda.synchronize()
            got += [q, k, cache.k_codes, cache.k_scales]
        return got
    for a, b in zip(steps(True), steps(False)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("which", ["prompt", "rope"])
def test_output_allocated_for_another_stream(which):
    """A call on a side stream that allocates its output does not write over memory that the
    current stream has freed but has yet to read."""
    hq, H, T = 16, 4, 100
    q, k, v = _inputs(T, hq, H, seed=25)
    cache = kvq.Cache.empty(128, H)
    pos = torch.arange(T).cuda()
    table = plain.rope_table(T, 128).cuda()
    cu = _cu([T])
    side = torch.cuda.Stream()
    kept = torch.zeros_like(q)
    old = torch.full_like(q, 3.0)
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)                      # some 50 ms
    kept.copy_(old)
    del old
    if which == "prompt":
        out = kvq.prompt_attention(q, k, v, cu, T, SCALE, stream=side)
    else:
        out = kvq.rope_quantize_scatter(cache, q, k, v, pos, table, pos, stream=side)
    torch.cuda.synchronize()
    assert torch.all(kept == 3.0)
    assert out.shape == q.shape


def test_a_serving_step_of_both_operators():
    """Prompts rotated in place and stored (kvq_rope_quantize_scatter), attended over
    (kvq_prompt_attention), then one decode step of new tokens: rotated, stored, and attended over
    the cache (kvq_paged_decode), each against the oracles."""
    hq, H, bs = 16, 4, 16
    lens = np.array([120, 33, 200], dtype=np.int32)
    T, N = int(lens.sum()), len(lens)
    q, k, v = _inputs(T, hq, H, seed=24)
    qf, kf, vf = (x.float().cpu().numpy() for x in (q, k, v))
    table = plain.rope_table(1024, 128)
    bt, blocks = workloads.block_tables(lens + 1, bs, 3, spare_blocks=2)
    slots = np.concatenate([workloads.token_slots(bt, r, int(L), bs) for r, L in enumerate(lens)])
    pos = np.concatenate([np.arange(L) for L in lens])
    cache = kvq.Cache.empty(blocks * bs, H, 128, bs)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()      # noqa: E731
    kvq.rope_quantize_scatter(cache, q, k, v, dev(pos), table.cuda(), dev(slots), q_out=q, k_out=k,
                              err_flags=err)
    out = kvq.prompt_attention(q, k, v, _cu(lens), int(lens.max()), SCALE, err_flags=err)
    # the decode step
    q1, k1, v1 = _inputs(N, hq, H, seed=25)
    new_slots = np.concatenate([workloads.token_slots(bt, r, int(L) + 1, bs)[-1:] for r, L in enumerate(lens)])
    q1r = kvq.rope_quantize_scatter(cache, q1, k1, v1, dev(lens.astype(np.int64)), table.cuda(),
                                    dev(new_slots), err_flags=err)
    got = kvq.paged_decode(cache, q1r, dev(bt), dev(lens + 1), int(lens.max()) + 1, SCALE, err_flags=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    # rotation of the prompts, then the attention over the rotated bf16 rows
    for x, xf in ((q, qf), (k, kf)):
        want = torch.from_numpy(plain.rotate_rows(xf, table.numpy(), pos, False)).to(torch.bfloat16)
        assert torch.equal(x.cpu(), want)
    assert_close(out, q, k, v, lens)
    # the cache, and the decode step over it
    oc = oracle.empty_cache(blocks * bs, H, 128)
    for at, kk, vv, pp in ((slots, kf, vf, pos),
                           (new_slots, k1.float().cpu().numpy(), v1.float().cpu().numpy(), lens)):
        rot = plain.rotate_rows(kk, table.numpy(), pp, False)
        oc["k_codes"][at], oc["k_scales"][at] = plain.quantize_f32_rows(rot)
        oc["v_codes"][at], oc["v_scales"][at] = plain.quantize_f32_rows(vv)
    for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
        assert np.array_equal(getattr(cache, name).cpu().numpy(), oc[name]), name
    want = torch.from_numpy(plain.rotate_rows(q1.float().cpu().numpy(), table.numpy(), lens, False)).to(torch.bfloat16)
    assert torch.equal(q1r.cpu(), want)
    ref, oerr = oracle.paged_attention(oc, workloads.bf16_bits(want), N, 1, hq, bt, lens + 1, bs, SCALE)
    assert oerr == 0
    assert_attention_close(got, ref, "decode after the rotary store")
