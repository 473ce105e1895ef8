"""The rotary store and the prompt attention: inputs, plain forms and calls, for measuring them.

Two operators of a serving step over the FP8 paged cache:

  rope    rotary position embedding of the step's query and key rows, the rotated keys and the
          values quantised (e4m3 codes, fp32 scale = row amax / 448) into their cache slots
  prompt  causal grouped-query attention of packed prompts over their own bf16 keys and values

With ``own`` False, ``run`` computes them with elementary torch operations in fp32, rounded once
at the end; with ``own`` True it calls this library.
"""
import math
import random

import numpy as np
import torch

own = False

D = 128


def listed():
    return [
        # One new token of one request: a decode step at batch 1, where latency counts.
        dict(name="rope_one_token", op="rope", tokens=1, pad=0, hq=32, h=8, rotary=128, interleaved=False,
             k_out=False, positions="decode", max_pos=8192, block=16),
        # A decode step of 32 requests whose contexts are 1,024 to 8,192 tokens long.
        dict(name="rope_decode_32", op="rope", tokens=32, pad=0, hq=32, h=8, rotary=128, interleaved=False,
             k_out=False, positions="decode", max_pos=8192, block=16),
        # A verify step: 64 requests, 4 rows each, far positions, the batch padded to a captured size.
        dict(name="rope_verify_64x4", op="rope", tokens=256, pad=11, hq=64, h=8, rotary=128, interleaved=False,
             k_out=False, positions="decode", max_pos=32768, block=64),
        # A prompt of odd length in a model that rotates half of each head, neighbouring dims paired.
        dict(name="rope_partial_1021", op="rope", tokens=1021, pad=0, hq=24, h=4, rotary=64, interleaved=True,
             k_out=True, positions="prompt", max_pos=4096, block=16),
        # Prompts of 16,384 tokens in all, queries and keys rotated for the prompt attention.
        dict(name="rope_prompts_16384", op="rope", tokens=16384, pad=0, hq=32, h=8, rotary=128, interleaved=False,
             k_out=True, positions="prompt", max_pos=8192, block=64),
        # One long prompt: a quarter of a 256K context in one call.
        dict(name="rope_long_65536", op="rope", tokens=65536, pad=0, hq=32, h=8, rotary=128, interleaved=False,
             k_out=True, positions="prompt", max_pos=65536, block=64),
        # A single short prompt: the smallest call.
        dict(name="prompt_one_64", op="prompt", n=1, lo=64, hi=64, tail=0, hq=32, h=8),
        # A batch of short ragged prompts (chat turns), the token buffer longer than they are.
        dict(name="prompt_short_batch", op="prompt", n=48, lo=1, hi=384, tail=37, hq=32, h=8),
        # One ordinary prompt of odd length, 7 query heads per KV head.
        dict(name="prompt_one_1999", op="prompt", n=1, lo=1999, hi=1999, tail=0, hq=28, h=4),
        # A ragged batch of ordinary prompts, 64 query heads.
        dict(name="prompt_batch_64_heads", op="prompt", n=8, lo=300, hi=4096, tail=0, hq=64, h=8),
        # Four requests of 8,192 tokens: a prefill batch.
        dict(name="prompt_4x8192", op="prompt", n=4, lo=8192, hi=8192, tail=0, hq=32, h=8),
        # One long prompt of odd length.
        dict(name="prompt_one_16381", op="prompt", n=1, lo=16381, hi=16381, tail=0, hq=32, h=8),
    ]


def _log_uniform(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


#: What a drawn case costs at most: the plain form's scores of the largest listed one.
_SCORES = 32 * 16381 * 16381


def draw(rng):
    h = rng.choice([1, 2, 4, 8])
    if rng.random() < 0.4:
        decode = rng.random() < 0.5
        tokens = _log_uniform(rng, 1, 512 if decode else 50000)
        return dict(op="rope", tokens=tokens, pad=rng.randint(0, max(0, tokens // 8)), hq=h * rng.choice([1, 2, 3, 4, 7, 8]),
                    h=h, rotary=rng.choice([128, 128, 64, 32, 96, 16]), interleaved=rng.random() < 0.3,
                    k_out=not decode, positions="decode" if decode else "prompt",
                    max_pos=max(tokens, rng.choice([4096, 8192, 32768, 131072])), block=rng.choice([16, 64]))
    hq = h * rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    n = _log_uniform(rng, 1, 64)
    most = min(16000, int(math.sqrt(_SCORES / (n * hq))))
    hi = _log_uniform(rng, 1, most)
    lo = hi if rng.random() < 0.3 else rng.randint(1, hi)
    return dict(op="prompt", n=n, lo=lo, hi=hi, tail=rng.choice([0, 0, 1, rng.randint(1, 300)]), hq=hq, h=h)


def _lens(case):
    """The prompts' lengths, the longest of them the case's bound."""
    n, lo, hi = case["n"], case["lo"], case["hi"]
    r = random.Random("%d %d %d" % (n, lo, hi))
    lens = [_log_uniform(r, lo, hi) for _ in range(n)]
    lens[r.randrange(n)] = hi
    return lens


def _positions(case, g):
    """Positions of the call's tokens: one per decoding request, or packed prompts from 0 up."""
    t, p = case["tokens"], case["max_pos"]
    if case["positions"] == "decode":
        return torch.randint(p // 8, p, (t,), generator=g)
    parts, left = [], t
    while left:
        n = min(left, int(torch.randint(p // 4, p + 1, (1,), generator=g)))
        parts.append(torch.arange(n))
        left -= n
    return torch.cat(parts)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    c = torch.Generator().manual_seed(int(seed))
    hq, h = case["hq"], case["h"]
    if case["op"] == "rope":
        t, r = case["tokens"], case["rotary"]
        # the projections' fused output; q, k and v are views of it
        qkv = torch.randn(t, (hq + 2 * h) * D, generator=g, device="cuda").to(torch.bfloat16)
        q = qkv[:, :hq * D].view(t, hq, D)
        k = qkv[:, hq * D:(hq + h) * D].view(t, h, D)
        v = qkv[:, (hq + h) * D:].view(t, h, D)
        angles = torch.arange(case["max_pos"], dtype=torch.float64, device="cuda")[:, None] * \
            10000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
        table = torch.cat([angles.cos(), angles.sin()], dim=1).to(torch.float32)
        # a cache somewhat larger than the call: other requests' rows stay as they are
        slots = ((t + t // 4 + 64) // case["block"] + 1) * case["block"]
        ids = torch.randperm(slots - 1, generator=c)[:t]
        if case["pad"]:
            ids[t - case["pad"]:] = -1                      # a padded batch: the last tokens are no tokens
        codes = [torch.randint(0, 0x7E, (slots, h, D), generator=g, device="cuda", dtype=torch.uint8) for _ in range(2)]
        scales = [torch.rand(slots, h, generator=g, device="cuda") / 448 for _ in range(2)]
        return dict(case=case, q=q, k=k, v=v, positions=_positions(case, c).cuda(), table=table, slots=ids.cuda(),
                    q_out=torch.zeros(t, hq, D, dtype=torch.bfloat16, device="cuda"),
                    k_out=torch.zeros(t, h, D, dtype=torch.bfloat16, device="cuda") if case["k_out"] else None,
                    k_codes=codes[0], v_codes=codes[1], k_scales=scales[0], v_scales=scales[1])
    lens = _lens(case)
    t = sum(lens) + case["tail"]
    # rotated queries and keys beside the values, as the projections leave them: views of one tensor
    qkv = torch.randn(t, (hq + 2 * h) * D, generator=g, device="cuda")
    qkv[:, :hq * D] *= 1.5                                   # scores of a spread of about 1.5
    qkv = qkv.to(torch.bfloat16)
    return dict(case=case, q=qkv[:, :hq * D].view(t, hq, D), k=qkv[:, hq * D:(hq + h) * D].view(t, h, D),
                v=qkv[:, (hq + h) * D:].view(t, h, D), max_len=max(lens), scale=1 / math.sqrt(D),
                cu=torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device="cuda"),
                out=torch.zeros(t, hq, D, dtype=torch.bfloat16, device="cuda"))


def _rotate(x, table, interleaved):
    """x [T, heads, D] in fp32, each pair of its first 2 n dims turned by its angle (table: n cosines, n sines)."""
    n = table.shape[1] // 2
    c, s = table[:, None, :n], table[:, None, n:]
    if interleaved:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        y = torch.stack([a * c - b * s, b * c + a * s], dim=-1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        y = torch.cat([a * c - b * s, b * c + a * s], dim=-1)
    return torch.cat([y, x[..., 2 * n:]], dim=-1)


def _store(codes, scales, rows, at, valid):
    """fp32 rows as e4m3 codes and scales into the slots `at`; rows that are not valid leave theirs as it was."""
    amax = rows.abs().amax(dim=-1)
    scale = amax / 448
    code = torch.where((amax > 0)[..., None], rows / scale[..., None], torch.zeros_like(rows)).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[at] = torch.where(valid[:, None, None], code, codes[at])
    scales[at] = torch.where(valid[:, None], scale, scales[at])


def _plain_rope(s):
    case = s["case"]
    valid = s["slots"] >= 0
    at = torch.where(valid, s["slots"], s["k_codes"].shape[0] - 1)   # the last slot is nobody's
    table = s["table"][s["positions"]]
    k = _rotate(s["k"].float(), table, case["interleaved"])
    q = _rotate(s["q"].float(), table, case["interleaved"])
    s["q_out"].copy_(torch.where(valid[:, None, None], q.to(torch.bfloat16), s["q_out"]))
    if s["k_out"] is not None:
        s["k_out"].copy_(torch.where(valid[:, None, None], k.to(torch.bfloat16), s["k_out"]))
    _store(s["k_codes"], s["k_scales"], k, at, valid)
    _store(s["v_codes"], s["v_scales"], s["v"].float(), at, valid)


def _plain_prompt(s):
    q, k, v, cu, out, length = s["q"], s["k"], s["v"], s["cu"], s["out"], s["max_len"]
    t, hq, h = q.shape[0], q.shape[1], k.shape[1]
    n, groups = cu.numel() - 1, hq // h
    # the prompts padded to the longest: [prompt, KV head, (query head,) position, dim]
    pos = torch.arange(length, device=q.device)
    rows = (cu[:-1, None] + pos).clamp(max=t - 1)
    qp = q[rows].float().view(n, length, h, groups, D).permute(0, 2, 3, 1, 4).reshape(n * h, groups * length, D)
    kp = k[rows].float().permute(0, 2, 1, 3).reshape(n * h, length, D)
    vp = v[rows].float().permute(0, 2, 1, 3).reshape(n * h, length, D)
    score = torch.bmm(qp, kp.transpose(1, 2)).mul_(s["scale"])
    score.view(n * h, groups, length, length).masked_fill_(pos[None, :] > pos[:, None], -math.inf)
    score.sub_(score.amax(dim=-1, keepdim=True)).exp_()
    o = torch.bmm(score, vp).div_(score.sum(dim=-1, keepdim=True))
    o = o.view(n, h, groups, length, D).permute(0, 3, 1, 2, 4).reshape(n, length, hq, D)
    # back to the packed rows; rows behind the last prompt stay as they were
    token = torch.arange(t, device=q.device)
    of = torch.searchsorted(cu[1:].contiguous(), token.to(torch.int32), right=True).clamp(max=n - 1)
    packed = o[of, (token - cu[of]).clamp(max=length - 1)]
    out.copy_(torch.where((token < cu[-1])[:, None, None], packed.to(torch.bfloat16), out))


def run(state):
    s = state
    if s["case"]["op"] == "rope":
        if own:
            import fp8_paged_kv_kvq_gb300 as kvq
            cache = kvq.Cache(s["k_codes"], s["v_codes"], s["k_scales"], s["v_scales"], s["case"]["block"])
            kvq.rope_quantize_scatter(cache, s["q"], s["k"], s["v"], s["positions"], s["table"], s["slots"],
                                      layout=kvq.ROPE_INTERLEAVED if s["case"]["interleaved"] else kvq.ROPE_HALVES,
                                      q_out=s["q_out"], k_out=s["k_out"])
        else:
            _plain_rope(s)
        f8 = torch.float8_e4m3fn
        return dict(q_out=s["q_out"], k_out=s["k_out"], k_codes=s["k_codes"].view(f8), v_codes=s["v_codes"].view(f8),
                    k_scales=s["k_scales"], v_scales=s["v_scales"])
    if own:
        import fp8_paged_kv_kvq_gb300 as kvq
        kvq.prompt_attention(s["q"], s["k"], s["v"], s["cu"], s["max_len"], s["scale"], out=s["out"])
    else:
        _plain_prompt(s)
    return s["out"]


def work(case):
    hq, h = case["hq"], case["h"]
    if case["op"] == "rope":
        t, live = case["tokens"], case["tokens"] - case["pad"]
        rows = hq + 2 * h
        table = 4 * case["rotary"] * min(live, case["max_pos"])
        moved = live * (rows * 2 * D + (hq + (h if case["k_out"] else 0)) * 2 * D + 2 * h * (D + 4))
        return dict(bytes=moved + table + 16 * t, flops=live * ((hq + h) * 3 * case["rotary"] + 2 * h * 2 * D))
    lens = _lens(case)
    pairs = sum(n * (n + 1) // 2 for n in lens)
    return dict(bytes=sum(lens) * (2 * hq + 2 * h) * 2 * D + 4 * len(lens) + 4, flops=4 * D * hq * pairs)


# ---------------------------------------------------------------------------
# The definitions in 64 bits.


def _e4m3(y):
    """The e4m3 value nearest to y (64 bits), ties to the even mantissa, at most 448."""
    a = y.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign((a / step).round() * step, y)


def _exact_rope(s):
    case, n = s["case"], s["case"]["rotary"] // 2
    live = torch.nonzero(s["slots"] >= 0).flatten()
    at = s["slots"][live]
    turn = s["table"][s["positions"][live]].double()
    turn = torch.complex(turn[:, :n], turn[:, n:])[:, None]

    def turned(x):
        x = x[live].double()
        pairs = x[..., :2 * n].unflatten(-1, (n, 2)) if case["interleaved"] else \
            x[..., :2 * n].unflatten(-1, (2, n)).transpose(-1, -2)
        pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        pairs = pairs if case["interleaved"] else pairs.transpose(-1, -2)
        return torch.cat([pairs.flatten(-2), x[..., 2 * n:]], dim=-1)

    q, k, v = turned(s["q"]), turned(s["k"]), s["v"][live].double()
    got = dict(q_out=s["q_out"].double().index_copy(0, live, q), k_out=None)
    if case["k_out"]:
        got["k_out"] = s["k_out"].double().index_copy(0, live, k)
    for name, x in (("k", k), ("v", v)):
        scale = x.abs().amax(dim=-1) / 448.0
        code = _e4m3(x / scale.clamp(min=1e-300)[..., None])
        got[name + "_codes"] = s[name + "_codes"].view(torch.float8_e4m3fn).double().index_copy(0, at, code)
        got[name + "_scales"] = s[name + "_scales"].double().index_copy(0, at, scale)
    return got


def _exact_prompt(s):
    out = s["out"].double()
    groups = s["q"].shape[1] // s["k"].shape[1]
    bounds = s["cu"].tolist()
    for a, b in zip(bounds[:-1], bounds[1:]):
        for head in range(s["k"].shape[1]):
            k, v = s["k"][a:b, head].double(), s["v"][a:b, head].double()
            for first in range(a, b, 1024):
                last = min(b, first + 1024)
                q = s["q"][first:last, head * groups:(head + 1) * groups].double()
                seen = torch.arange(a, last, device=q.device)[None, :] <= torch.arange(first, last, device=q.device)[:, None]
                x = torch.einsum("qgd,kd->qgk", q, k[:last - a]) * s["scale"]
                w = torch.softmax(torch.where(seen[:, None, :], x, -math.inf), dim=-1)
                out[first:last, head * groups:(head + 1) * groups] = torch.einsum("qgk,kd->qgd", w, v[:last - a])
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_rope(s) if case["op"] == "rope" else _exact_prompt(s)
