"""Refusals of kvq_rope_quantize_scatter and kvq_prompt_attention: every call
here is answered on the host, before anything could be launched."""
import ctypes
import subprocess
import sys

import pytest
import torch

import fp8_paged_kv_kvq_gb300 as kvq
from fp8_paged_kv_kvq_gb300 import build as kbuild

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kvq.load()


def _cache(head_dim=128, ptr=0x10000, H=8):
    return kvq._CacheStruct(ptr, ptr + 0x100000, ptr + 0x200000, ptr + 0x300000, 64, H, head_dim, 16)


ROPE = dict(q=0x1000, qs=6144, hq=32, k=0x2000, ks=6144, v=0x3000, vs=6144, T=4, pos=0x4000,
            table=0x5000, P=128, r=128, layout=0, slots=0x6000, qo=0x7000, qos=4096, ko=0x8000,
            kos=1024, err=0)


def _rope(lib, cache="default", **changes):
    a = dict(ROPE, **changes)
    c = _cache() if cache == "default" else cache
    return lib.kvq_rope_quantize_scatter(
        None if c is None else ctypes.byref(c), P(a["q"]), a["qs"], a["hq"], P(a["k"]), a["ks"],
        P(a["v"]), a["vs"], a["T"], P(a["pos"]), P(a["table"]), a["P"], a["r"], a["layout"],
        P(a["slots"]), P(a["qo"]), a["qos"], P(a["ko"]), a["kos"], P(a["err"]), P(0))


@pytest.mark.parametrize("changes,status", [
    (dict(T=0), OK), (dict(T=0, q=0, k=0, v=0, pos=0, slots=0, qo=0, hq=0), OK),
    (dict(T=-1), INVALID), (dict(hq=-1), INVALID), (dict(P=-1), INVALID),
    (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(pos=0), INVALID), (dict(slots=0), INVALID),
    (dict(table=0), INVALID), (dict(q=0), INVALID), (dict(qo=0), INVALID), (dict(hq=0), INVALID),
    (dict(q=0, qo=0), INVALID), (dict(layout=2), INVALID), (dict(layout=-1), INVALID),
    (dict(r=0), INVALID), (dict(r=-16), INVALID), (dict(r=144), INVALID), (dict(r=8), UNSUPPORTED),
    (dict(r=100), UNSUPPORTED), (dict(qs=-8), INVALID), (dict(kos=-8), INVALID),
    (dict(qs=6148), MISALIGNED), (dict(ks=6148), MISALIGNED), (dict(vs=6148), MISALIGNED),
    (dict(qos=4100), MISALIGNED), (dict(kos=1028), MISALIGNED), (dict(q=0x1008), MISALIGNED),
    (dict(k=0x2008), MISALIGNED), (dict(v=0x3004), MISALIGNED), (dict(qo=0x7002), MISALIGNED),
    (dict(ko=0x8004), MISALIGNED), (dict(table=0x5004), MISALIGNED), (dict(pos=0x4004), MISALIGNED),
    (dict(slots=0x6004), MISALIGNED), (dict(err=2), MISALIGNED),
    (dict(qos=4088), INVALID), (dict(kos=1016), INVALID),       # output rows that overlap
    (dict(qo=0x1000, qos=4096), INVALID),                       # in place with another stride
    (dict(ko=0x2000, kos=1024), INVALID),
    (dict(T=1 << 30), UNSUPPORTED),                             # rows numbered in 32 bits
])
def test_rope_refusals(lib, changes, status):
    assert _rope(lib, **changes) == status


def test_rope_cache_refusals(lib):
    assert _rope(lib, cache=None) == INVALID
    assert _rope(lib, cache=_cache(head_dim=64), r=64) == UNSUPPORTED
    assert _rope(lib, cache=_cache(ptr=0x10008)) == MISALIGNED


PROMPT = dict(q=0x1000, qs=6144, k=0x2000, ks=6144, v=0x3000, vs=6144, T=100, cu=0x4000, N=3,
              most=64, hq=32, h=8, d=128, scale=0.1, out=0x5000, os=4096, err=0)


def _prompt(lib, **changes):
    a = dict(PROMPT, **changes)
    return lib.kvq_prompt_attention(P(a["q"]), a["qs"], P(a["k"]), a["ks"], P(a["v"]), a["vs"],
                                    a["T"], P(a["cu"]), a["N"], a["most"], a["hq"], a["h"], a["d"],
                                    a["scale"], P(a["out"]), a["os"], P(a["err"]), P(0))


@pytest.mark.parametrize("changes,status", [
    (dict(T=0), OK), (dict(N=0), OK), (dict(T=0, q=0, k=0, v=0, out=0, cu=0), OK),
    (dict(T=-1), INVALID), (dict(N=-1), INVALID), (dict(most=-1), INVALID), (dict(hq=0), INVALID),
    (dict(h=0), INVALID), (dict(hq=30), INVALID), (dict(d=0), INVALID),
    (dict(scale=0.0), INVALID), (dict(scale=-0.1), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(scale=float("inf")), INVALID), (dict(d=64), UNSUPPORTED),
    (dict(hq=8 * 129, qs=8 * 129 * 128, os=8 * 129 * 128), UNSUPPORTED),
    (dict(qs=1 << 40), UNSUPPORTED), (dict(ks=1 << 40), UNSUPPORTED), (dict(vs=1 << 40), UNSUPPORTED),
    (dict(T=1 << 31), UNSUPPORTED), (dict(N=0x7FFFFFFE), UNSUPPORTED),
    (dict(qs=4088), INVALID), (dict(ks=1016), INVALID), (dict(vs=1016), INVALID),
    (dict(os=4088), INVALID), (dict(q=0), INVALID), (dict(k=0), INVALID), (dict(v=0), INVALID),
    (dict(out=0), INVALID), (dict(cu=0), INVALID), (dict(qs=6148), MISALIGNED),
    (dict(ks=6148), MISALIGNED), (dict(vs=6148), MISALIGNED), (dict(os=4100), MISALIGNED),
    (dict(q=0x1008), MISALIGNED), (dict(k=0x2008), MISALIGNED), (dict(v=0x3008), MISALIGNED),
    (dict(out=0x5008), MISALIGNED), (dict(cu=0x4002), MISALIGNED), (dict(err=2), MISALIGNED),
])
def test_prompt_refusals(lib, changes, status):
    assert _prompt(lib, **changes) == status


def test_bindings_reject_bad_tensors():
    """dtypes, shapes, layouts and devices are checked before the library is called."""
    bf = torch.bfloat16
    q, k, v = torch.zeros(4, 8, 128, dtype=bf), torch.zeros(4, 2, 128, dtype=bf), \
        torch.zeros(4, 2, 128, dtype=bf)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    for args in ((q.float(), k, v, cu), (q, k[:3], v, cu), (q, k, v[:, :1], cu),
                 (q, k, v, cu.long()), (q, k, v, cu[None]), (q, k, v, cu[:0]),
                 (q.transpose(0, 1), k, v, cu), (q[:, :, ::2], k[:, :, ::2], v[:, :, ::2], cu)):
        with pytest.raises(ValueError):
            kvq.prompt_attention(*args, 4, 0.1)
    with pytest.raises(ValueError):
        kvq.prompt_attention(q, k, v, cu, 4, 0.1, out=torch.zeros(4, 4, 128, dtype=bf))
    with pytest.raises(ValueError):
        kvq.prompt_attention(q, k, v, cu, 4, 0.1, err_flags=torch.zeros(1))
    with pytest.raises(ValueError, match="current CUDA device"):
        kvq.prompt_attention(q, k, v, cu, 4, 0.1)                # host tensors

    cache = kvq.Cache.empty(64, 2, 128, 16, device="cpu")
    pos, slots, table = torch.arange(4), torch.arange(4), torch.zeros(16, 128)
    good = dict(q=q, k=k, v=v, positions=pos, rope_table=table, slot_ids=slots)
    for bad in (dict(q=q.float()), dict(k=k[:, :1]), dict(v=v[:3]), dict(positions=pos.int()),
                dict(positions=pos[:3]), dict(slot_ids=slots.int()), dict(rope_table=table.double()),
                dict(rope_table=table[0]), dict(rope_table=table[:, ::2]), dict(q_out=q[:, :4]),
                dict(q=None, q_out=q), dict(k_out=k[:3]), dict(err_flags=torch.zeros(1)),
                dict(q=q[:, :, :64])):
        with pytest.raises(ValueError):
            kvq.rope_quantize_scatter(cache, **{**good, **bad})
    with pytest.raises(ValueError, match="current CUDA device"):
        kvq.rope_quantize_scatter(cache, **good)


def test_binding_without_private_torch_calls():
    """The current stream and device come from public calls where torch lacks its private ones:
    the package is imported by a torch without them, and the binding asks those."""
    code = """
import types, torch
for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"):
    if hasattr(torch._C, name):
        delattr(torch._C, name)
torch.cuda.is_initialized = lambda: True
torch.cuda.current_device = lambda: -1            # (a host tensor's)
torch.cuda.current_stream = lambda d: types.SimpleNamespace(cuda_stream=0x1230 + d)
import fp8_paged_kv_kvq_gb300 as kvq
assert kvq._one_device([torch.zeros(1), None]) == -1
assert kvq._raw_stream(None, 4) == 0x1234
side = types.SimpleNamespace(device_index=4, cuda_stream=0x4000)
assert kvq._raw_stream(side, 4) == 0x4000
try:
    kvq._raw_stream(side, 3)
except ValueError:
    print("refused")
"""
    res = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                         cwd=kbuild.ROOT)
    assert res.returncode == 0 and "refused" in res.stdout, res.stderr
