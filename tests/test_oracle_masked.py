"""Pins of oracle/masked.py: worked masks, the dense causal oracle, a pool by hand."""
import torch

import oracle.masked as plain


def test_window_rule_by_hand():
    see = plain.window_rule(3, 1)(6, 2, 0).int().tolist()
    assert see == [[1, 0, 1, 1, 1, 0], [1, 0, 0, 1, 1, 1]]
    assert plain.window_rule(1, 0)(2, 3, 0).int().tolist() == [[0, 0], [1, 0], [0, 1]]


def test_tree_rule_by_hand():
    # two roots, node 2 on node 0; the bit of a node that does not exist is ignored
    mask = torch.tensor([[[0b0001], [0b1010], [0b0101]]], dtype=torch.int32)
    assert plain.tree_rule(mask)(5, 3, 0).int().tolist() == [[1, 1, 1, 0, 0], [1, 1, 0, 1, 0], [1, 1, 1, 0, 1]]
    assert plain.tree_rule(mask)(2, 3, 0).int().tolist() == [[0, 0], [1, 0], [0, 1]]


def _cache(slots, H, seed):
    g = torch.Generator().manual_seed(seed)
    x = [torch.randn(slots, H, 128, generator=g) for _ in range(2)]
    s = [t.abs().amax(-1) / 448 for t in x]
    c = [(t / u[..., None]).to(torch.float8_e4m3fn) for t, u in zip(x, s)]
    return dict(k_codes=c[0], v_codes=c[1], k_scales=s[0], v_scales=s[1], block_size=16)


def test_wide_window_is_causal_attention():
    H, Hq, R, L = 2, 4, 3, 37
    c = _cache(48, H, 1)
    q = torch.randn(R, Hq, 128, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    tables = torch.tensor([[2, 0, 1]], dtype=torch.int32)
    out = plain.attention(c, q, tables, [L], R, 0.09, plain.window_rule(100, 0))[0]
    lower = torch.tensor([[0b001], [0b011], [0b111]], dtype=torch.int32)[None]
    out_tree = plain.attention(c, q, tables, [L], R, 0.09, plain.tree_rule(lower))[0]
    slot = torch.cat([torch.arange(32, 48), torch.arange(0, 16), torch.arange(16, 32)])[:L]
    k = (c["k_codes"].double() * c["k_scales"].double()[..., None])[slot].repeat_interleave(2, 1)
    v = (c["v_codes"].double() * c["v_scales"].double()[..., None])[slot].repeat_interleave(2, 1)
    see = torch.arange(L)[None] <= torch.arange(L - R, L)[:, None]
    ref = torch.nn.functional.scaled_dot_product_attention(
        q.double().transpose(0, 1), k.transpose(0, 1), v.transpose(0, 1), attn_mask=see, scale=0.09)
    assert torch.allclose(out, ref.transpose(0, 1), rtol=1e-12, atol=1e-12)
    assert torch.allclose(out_tree, out, rtol=1e-12, atol=1e-12)


def test_pool_by_hand():
    p = plain.Pool(6)
    tables = [[-1] * 4, [-1] * 4]
    p.alloc(tables, [0, 0], [2, 1])
    assert tables == [[5, 4, -1, -1], [3, -1, -1, -1]] and p.free == [0, 1, 2]
    child = [[-1] * 4 for _ in range(3)]
    lens, copies = p.fork([0, 0, 1], tables, [20, 16], child, 16)
    assert lens == [20, 20, 16] and copies == [(64, 32, 4), (64, 16, 4)]
    assert child == [[5, 2, -1, -1], [5, 1, -1, -1], [3, -1, -1, -1]]
    assert p.refs == [0, 1, 1, 2, 1, 3] and p.free == [0]
    p.release(tables, [0, 0], [2, 1])
    assert p.refs == [0, 1, 1, 1, 0, 2] and p.free == [0, 4]
    p.alloc(child, [2, 2, 1], [3, 3, 2])
    assert [row[2] for row in child[:2]] == [4, 0] and child[2][1] == -1 and p.free == []
