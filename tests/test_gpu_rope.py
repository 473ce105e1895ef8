"""kvq_rope_quantize_scatter on the GPU.

Codes and scales must equal, bit for bit, the binary32 evaluation of the
rotation and the row codec (oracle/prompt.py); q_out and k_out must equal that
rotation rounded to bf16.  Against the rotation in 64 bits, a rotated value
carries two products and a sum rounded to binary32, each by at most 2^-24 of
its result, so at most 2^-22 (|a| + |b|) in all, and q_out one bf16 rounding
(2^-8 of the value) more; a cached value one e4m3 rounding (2^-4 of the value,
or half a subnormal step, 2^-10 of the scale) and the quotient's (2^-22)."""
import numpy as np
import pytest
import torch

import fp8_paged_kv_kvq_gb300 as kvq
import oracle
import oracle.prompt as plain
import workloads

pytestmark = pytest.mark.gpu


def _inputs(T, hq, H, seed, scale=1.0):
    """q, k, v as views of one fused projection output on the GPU."""
    g = workloads.generator(seed, 201)
    qkv = (torch.randn(T, (hq + 2 * H) * 128, generator=g) * scale).to(torch.bfloat16).cuda()
    return (qkv, qkv[:, :hq * 128].view(T, hq, 128), qkv[:, hq * 128:(hq + H) * 128].view(T, H, 128),
            qkv[:, (hq + H) * 128:].view(T, H, 128))


def _f32(x):
    return x.float().cpu().numpy()


def _cache(slots, H, seed=5):
    """A cache that holds other requests' rows (random codes and scales)."""
    c = kvq.Cache.empty(slots, H, 128, 16)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for x in (c.k_codes, c.v_codes):
        x.copy_(torch.randint(0, 0x7E, x.shape, generator=g, device="cuda", dtype=torch.uint8))
    for x in (c.k_scales, c.v_scales):
        x.copy_(torch.rand(x.shape, generator=g, device="cuda"))
    return c


def _planes(c):
    return [x.cpu().numpy().copy() for x in (c.k_codes, c.v_codes, c.k_scales, c.v_scales)]


def _check(cache, before, kf, vf, slots, table, pos, interleaved, k_out=None, q=None, q_out=None):
    """The cache's planes, k_out and q_out against the plain forms; other slots as `before`."""
    rot = plain.rotate_rows(kf, table, pos, interleaved)
    live = slots >= 0
    want = [x.copy() for x in before]
    for i, rows in ((0, rot), (1, vf)):
        codes, scales = plain.quantize_f32_rows(rows)
        want[i][slots[live]] = codes[live]
        want[i + 2][slots[live]] = scales[live]
    got = _planes(cache)
    for i, name in enumerate(("k_codes", "v_codes", "k_scales", "v_scales")):
        a, b = got[i], want[i]
        if a.dtype == np.float32:
            a, b = a.view(np.uint32), b.view(np.uint32)
        assert np.array_equal(a, b), f"{name}: {(a != b).sum()} of {a.size} differ"
    # against 64 bits
    n = table.shape[1] // 2
    mag = np.abs(kf).astype(np.float64)
    i0, i1 = plain._pairs(2 * n, interleaved)
    pair = np.zeros_like(mag)
    pair[..., i0] = pair[..., i1] = mag[..., i0] + mag[..., i1]
    r64 = plain.rotate_rows64(kf, table, pos, interleaved)
    value = oracle.e4m3_decode(got[0][slots[live]].reshape(-1)).reshape(r64[live].shape) * \
        got[2][slots[live]].astype(np.float64)[..., None]
    tol = (2.0 ** -4 + 2.0 ** -22) * np.abs(r64[live]) + 2.0 ** -21 * pair[live] + \
        2.0 ** -10 * got[2][slots[live]].astype(np.float64)[..., None]
    assert np.all(np.abs(value - r64[live]) <= tol)
    for x, y in ((kf, k_out), (q, q_out)):
        if y is None:
            continue
        want_bf = torch.from_numpy(plain.rotate_rows(x, table, pos, interleaved)).to(torch.bfloat16)
        idx = torch.from_numpy(np.flatnonzero(live))
        assert torch.equal(y.cpu()[idx].view(torch.int16), want_bf[idx].view(torch.int16))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,hq,H,r", [
    (1, 32, 8, 128), (3, 8, 8, 64), (33, 7, 1, 128), (130, 28, 4, 96), (257, 5, 5, 32),
    (64, 24, 8, 16), (19, 16, 2, 112), (1021, 12, 4, 80),
])
def test_codes_and_rows_match_the_plain_forms(T, hq, H, r, interleaved):
    _, q, k, v = _inputs(T, hq, H, seed=T + r)
    table = plain.rope_table(4096, r)
    g = workloads.generator(T, 7)
    pos = torch.randint(0, 4096, (T,), generator=g)
    slots = torch.randperm(T + 9, generator=g)[:T]
    cache = _cache(T + 9, H)
    before = _planes(cache)
    k_out = torch.zeros(T, H, 128, dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    q_out = kvq.rope_quantize_scatter(cache, q, k, v, pos.cuda(), table.cuda(), slots.cuda(),
                                      layout=int(interleaved), k_out=k_out, err_flags=err)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    _check(cache, before, _f32(k), _f32(v), slots.numpy(), table.numpy(), pos.numpy(), interleaved,
           k_out, _f32(q), q_out)
    # the bf16 rows against 64 bits
    r64 = plain.rotate_rows64(_f32(q), table.numpy(), pos.numpy(), interleaved)
    x = np.abs(_f32(q)).astype(np.float64)
    i0, i1 = plain._pairs(r, interleaved)
    x[..., i0] = x[..., i1] = x[..., i0] + x[..., i1]
    assert np.all(np.abs(_f32(q_out) - r64) <= 2.0 ** -8 * np.abs(r64) + 2.0 ** -21 * x)


@pytest.mark.parametrize("r,interleaved", [(128, False), (64, False), (32, False), (128, True)])
def test_rotation_in_place(r, interleaved):
    """q_out = q and k_out = k, strided views of the fused output; v stays."""
    T, hq, H = 203, 16, 4
    qkv, q, k, v = _inputs(T, hq, H, seed=3)
    qf, kf, vf = _f32(q), _f32(k), _f32(v)
    table = plain.rope_table(512, r)
    pos = torch.arange(T) + 100
    slots = torch.arange(T) * 2
    cache = _cache(2 * T, H)
    before = _planes(cache)
    kvq.rope_quantize_scatter(cache, q, k, v, pos.cuda(), table.cuda(), slots.cuda(),
                              layout=int(interleaved), q_out=q, k_out=k)
    torch.cuda.synchronize()
    _check(cache, before, kf, vf, slots.numpy(), table.numpy(), pos.numpy(), interleaved, k, qf, q)
    assert np.array_equal(_f32(v), vf)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("T", [700, 1301])
@pytest.mark.parametrize("r,interleaved", [(128, False), (64, False), (32, False), (96, False),
                                           (16, False), (128, True), (80, True)])
def test_calls_of_many_tokens(r, interleaved, T, in_place):
    """More tokens than SMs have warps for their rows: a token's rows one after the other on two
    warps (700 tokens) or one, the next fetched ahead -- in place too, where a row fetched ahead
    must be one that nobody has rotated."""
    hq, H = 32, 8
    _, q, k, v = _inputs(T, hq, H, seed=T + r)
    qf, kf, vf = _f32(q), _f32(k), _f32(v)
    table = plain.rope_table(2048, r)
    g = workloads.generator(T, r)
    pos = torch.randint(0, 2048, (T,), generator=g)
    slots = torch.randperm(T + 5, generator=g)[:T]
    slots[T // 2] = -1
    cache = _cache(T + 5, H)
    before = _planes(cache)
    outs = dict(q_out=q, k_out=k) if in_place else \
        dict(q_out=torch.full((T, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda"),
             k_out=torch.full((T, H, 128), 7.0, dtype=torch.bfloat16, device="cuda"))
    kvq.rope_quantize_scatter(cache, q, k, v, pos.cuda(), table.cuda(), slots.cuda(),
                              layout=int(interleaved), **outs)
    torch.cuda.synchronize()
    _check(cache, before, kf, vf, slots.numpy(), table.numpy(), pos.numpy(), interleaved,
           outs["k_out"], qf, outs["q_out"])
    for name, x in (("q_out", qf), ("k_out", kf)):       # the skipped token's rows
        want = x[T // 2] if in_place else np.full_like(x[T // 2], 7.0)
        assert np.array_equal(_f32(outs[name])[T // 2], want)
    assert np.array_equal(_f32(v), vf)


def test_rotation_zero_is_the_plain_store():
    """Position 0 (cosines 1, sines 0): codes and scales are kvq_quantize_scatter's of the same
    rows -- large and tiny rows, all-zero rows, negative zeros and rows of subnormals among them."""
    T, H = 96, 4
    _, _, k, v = _inputs(T, 1, H, seed=8)
    k, v = k.contiguous(), v.contiguous()
    mags = torch.tensor([1.0, 3e37, 1e-30, 2.0 ** -120, 2.0 ** -133, 0.0, -0.0, 448.0]).cuda()
    for x in (k, v):
        x.mul_(mags.repeat(T // 8)[:, None, None].to(torch.bfloat16))
    x = torch.zeros_like(k)
    x[:, :, ::3] = -0.0
    k[5::16] = x[5::16]
    v[1, :, 5:] = -0.0
    slots = torch.randperm(T, generator=workloads.generator(1, 2)).cuda()
    a, b = _cache(T, H), _cache(T, H)
    table = torch.cat([torch.ones(1, 64), torch.zeros(1, 64)], dim=1).cuda()
    kvq.rope_quantize_scatter(a, None, k, v, torch.zeros(T, dtype=torch.int64, device="cuda"), table,
                              slots)
    kvq.quantize_scatter(b, k, v, slots)
    torch.cuda.synchronize()
    for i, (x, y) in enumerate(zip(_planes(a), _planes(b))):
        if i == 0:
            # (a 1 - b 0 of a zero a may change the zero's sign: compare K's values)
            x, y = oracle.e4m3_decode(x.reshape(-1)), oracle.e4m3_decode(y.reshape(-1))
        assert np.array_equal(x, y)


@pytest.mark.parametrize("T", [32, 1301])
def test_rows_that_are_not_finite_are_stored_as_the_store_stores_them(T):
    """A NaN or an infinity anywhere in a value row, or in a key's dims that are not rotated, gives
    the codes and the NaN scale of kvq_quantize_scatter, so that the row reads back as NaN; one in
    the rotated dims, or a rotation that leaves binary32, gives a NaN scale too; other rows stay
    finite."""
    H = 8
    inf, nan = float("inf"), float("nan")
    _, q, k, v = _inputs(T, 8, H, seed=31)
    k, v = k.contiguous(), v.contiguous()
    every = torch.tensor([nan, -nan] * 64, dtype=torch.bfloat16, device="cuda")
    for x in (k, v):
        x[1, 2, 20:] = every[20:]
        for token, head, dim, bad in ((3, 0, 77, nan), (4, 7, 127, -nan), (5, 1, 20, inf),
                                      (6, 3, 99, -inf), (7, 5, 64, inf), (7, 5, 65, nan)):
            x[token, head, dim] = bad
    v[9, 4] = every                                     # a row of nothing else
    v[10, 6, 0], v[11, 6, 3] = nan, inf
    slots = torch.randperm(T, generator=workloads.generator(31, T)).cuda()
    table = torch.cat([torch.ones(1, 8), torch.zeros(1, 8)], dim=1).cuda()      # no turn
    pos = torch.zeros(T, dtype=torch.int64, device="cuda")
    a, b = _cache(T, H), _cache(T, H)
    kvq.rope_quantize_scatter(a, q, k, v, pos, table, slots)
    kvq.quantize_scatter(b, k, v, slots)
    torch.cuda.synchronize()
    got, want = _planes(a), _planes(b)
    for x, y in zip(got[:2], want[:2]):
        assert np.array_equal(x, y)
    for x, y, rows in zip(got[2:], want[2:], (6, 9)):
        assert np.isnan(y).sum() == rows                # the existing store's NaN scales
        assert np.array_equal(x, y, equal_nan=True)

    k2 = k.clone()
    k2[:, :, 16:] = 1.0
    k2[12, 0, 3], k2[13, 1, 5] = nan, inf
    k2[14, 2, :16] = 3.0e38                             # a c + b s beyond FLT_MAX
    turn = torch.full((1, 16), 0.5 ** 0.5, device="cuda")
    for layout in (kvq.ROPE_HALVES, kvq.ROPE_INTERLEAVED):
        kvq.rope_quantize_scatter(a, q, k2, v, pos, turn, slots, layout=layout)
        torch.cuda.synchronize()
        scales = a.k_scales[slots].isnan().cpu()
        bad = torch.zeros(T, H, dtype=torch.bool)
        bad[12, 0] = bad[13, 1] = bad[14, 2] = True
        assert torch.equal(scales, bad)


def test_skipped_tokens_leave_everything_as_it_was():
    """Padding (slot -1, whatever its position), slots and positions out of range: flagged where
    out of range; their q_out, k_out and cache rows stay; the other tokens are stored."""
    T, hq, H = 40, 8, 2
    _, q, k, v = _inputs(T, hq, H, seed=9)
    table = plain.rope_table(64, 128)
    pos = torch.arange(T)
    slots = torch.arange(T)
    slots[30:] = -1
    pos[30:35] = 1 << 40                       # padding: not looked at
    kw = dict(q_out=torch.full((T, hq, 128), 7.0, dtype=torch.bfloat16, device="cuda"),
              k_out=torch.full((T, H, 128), 7.0, dtype=torch.bfloat16, device="cuda"))
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cache = _cache(64, H)
    before = _planes(cache)
    kvq.rope_quantize_scatter(cache, q, k, v, pos.cuda(), table.cuda(), slots.cuda(), err_flags=err,
                              **kw)
    torch.cuda.synchronize()
    assert int(err.item()) == 0
    safe = np.where(slots.numpy() >= 0, pos.numpy(), 0)
    _check(cache, before, _f32(k), _f32(v), slots.numpy(), table.numpy(), safe, False, kw["k_out"],
           _f32(q), kw["q_out"])
    assert torch.all(kw["q_out"][30:] == 7) and torch.all(kw["k_out"][30:] == 7)
    for change, flag in (((slots, 3, 64), kvq.ERRF_SLOT_RANGE), ((slots, 3, 1 << 62), kvq.ERRF_SLOT_RANGE),
                         ((pos, 4, 64), kvq.ERRF_POSITION_RANGE), ((pos, 4, -1), kvq.ERRF_POSITION_RANGE),
                         ((pos, 4, 1 << 60), kvq.ERRF_POSITION_RANGE)):
        p2, s2 = pos.clone(), slots.clone()
        (s2 if change[0] is slots else p2)[change[1]] = change[2]
        cache = _cache(64, H)
        before = _planes(cache)
        err.zero_()
        for x in kw.values():
            x.fill_(7.0)
        kvq.rope_quantize_scatter(cache, q, k, v, p2.cuda(), table.cuda(), s2.cuda(), err_flags=err,
                                  **kw)
        torch.cuda.synchronize()
        assert int(err.item()) == flag
        s2[change[1]] = -1
        p2[s2 < 0] = 0
        _check(cache, before, _f32(k), _f32(v), s2.numpy(), table.numpy(), p2.numpy(), False,
               kw["k_out"], _f32(q), kw["q_out"])
        assert torch.all(kw["q_out"][change[1]] == 7) and torch.all(kw["k_out"][change[1]] == 7)


def test_slots_past_32_bit_offsets():
    """A cache of 5 GB planes: slots whose code offsets pass 2^32 bytes."""
    H, S, T = 8, 5_000_000, 64
    _, q, k, v = _inputs(T, 8, H, seed=10)
    cache = kvq.Cache.empty(S, H, 128, 16)
    slots = S - 1 - 3 * torch.arange(T)
    slots[::7] = 11 + torch.arange(len(slots[::7]))
    table = plain.rope_table(131072, 128)
    pos = 131071 - torch.arange(T)
    q_out = kvq.rope_quantize_scatter(cache, q, k, v, pos.cuda(), table.cuda(), slots.cuda())
    torch.cuda.synchronize()
    small = kvq.Cache(*(x[slots.cuda()].clone() for x in (cache.k_codes, cache.v_codes,
                                                           cache.k_scales, cache.v_scales)), 16)
    zeros = [np.zeros_like(x) for x in _planes(small)]
    _check(small, zeros, _f32(k), _f32(v), np.arange(T), table.numpy(), pos.numpy(), False, None,
           _f32(q), q_out)
    written = int((cache.k_scales > 0).sum())
    assert written == T * H


def test_captured_replayed_and_on_another_stream():
    """A captured call replayed on new rows, positions and slots, and a call on a stream that the
    inputs do not come from."""
    T, hq, H = 48, 16, 4
    table = plain.rope_table(256, 128)
    qkv, q, k, v = _inputs(T, hq, H, seed=21)
    pos, slots = torch.arange(T).cuda(), torch.arange(T).cuda()
    q_out = torch.zeros(T, hq, 128, dtype=torch.bfloat16, device="cuda")
    cache = _cache(128, H)
    dev_table = table.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        kvq.rope_quantize_scatter(cache, q, k, v, pos, dev_table, slots, q_out=q_out)
    for seed in (22, 23):
        new, _, _, _ = _inputs(T, hq, H, seed=seed)
        qkv.copy_(new)
        pos.copy_(torch.randint(0, 256, (T,), generator=workloads.generator(seed, 1)))
        slots.copy_(torch.randperm(128, generator=workloads.generator(seed, 2))[:T])
        before = _planes(cache)
        graph.replay()
        torch.cuda.synchronize()
        _check(cache, before, _f32(k), _f32(v), slots.cpu().numpy(), table.numpy(),
               pos.cpu().numpy(), False, None, _f32(q), q_out)
    before = _planes(cache)
    q_out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    kvq.rope_quantize_scatter(cache, q, k, v, pos, dev_table, slots, q_out=q_out, stream=side)
    side.synchronize()
    _check(cache, before, _f32(k), _f32(v), slots.cpu().numpy(), table.numpy(), pos.cpu().numpy(),
           False, None, _f32(q), q_out)


def test_empty_call():
    cache = _cache(16, 2)
    before = _planes(cache)
    z = torch.zeros(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    out = kvq.rope_quantize_scatter(cache, z, z, z, none, plain.rope_table(4, 128).cuda(), none)
    torch.cuda.synchronize()
    assert out.shape == z.shape
    assert all(np.array_equal(a, b) for a, b in zip(before, _planes(cache)))
