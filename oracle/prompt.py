"""The rotary store and the prompt attention in plain form -- TEST INFRASTRUCTURE ONLY.

``rotate_rows`` and ``quantize_f32_rows`` evaluate the rotation and the row
codec one binary32 operation at a time with numpy (every product, sum and
quotient rounded once), so codes and scales must match bit for bit;
``rotate_rows64`` is the same rotation in 64 bits, written as a complex product.
``prompt_attention`` is causal grouped-query attention of packed sequences as
dense fp64 matrix products, with the magnitudes that its error bound needs."""
from __future__ import annotations

import numpy as np
import torch

from . import e4m3_encode


def rope_table(num_positions: int, rotary_dim: int, theta: float = 10000.0) -> torch.Tensor:
    """fp32 [num_positions, rotary_dim]: cosines then sines of p theta^(-2i/rotary_dim)."""
    i = np.arange(0, rotary_dim, 2, dtype=np.float64)
    a = np.arange(num_positions, dtype=np.float64)[:, None] * theta ** (-i / rotary_dim)
    return torch.from_numpy(np.concatenate([np.cos(a), np.sin(a)], axis=1).astype(np.float32))


def _pairs(r: int, interleaved: bool):
    n = r // 2
    return (np.arange(0, r, 2), np.arange(1, r, 2)) if interleaved else \
        (np.arange(n), np.arange(n, r))


def rotate_rows(x: np.ndarray, table: np.ndarray, positions: np.ndarray,
                interleaved: bool) -> np.ndarray:
    """x float32 [T, heads, D] rotated in binary32, one rounding per operation."""
    assert x.dtype == np.float32 and table.dtype == np.float32
    n = table.shape[1] // 2
    i0, i1 = _pairs(2 * n, interleaved)
    c, s = table[positions][:, None, :n], table[positions][:, None, n:]
    y = x.copy()
    y[..., i0] = x[..., i0] * c - x[..., i1] * s
    y[..., i1] = x[..., i1] * c + x[..., i0] * s
    return y


def rotate_rows64(x: np.ndarray, table: np.ndarray, positions: np.ndarray,
                  interleaved: bool) -> np.ndarray:
    n = table.shape[1] // 2
    i0, i1 = _pairs(2 * n, interleaved)
    t = table[positions].astype(np.float64)
    z = (x[..., i0].astype(np.float64) + 1j * x[..., i1]) * (t[:, None, :n] + 1j * t[:, None, n:])
    y = x.astype(np.float64)
    y[..., i0], y[..., i1] = z.real, z.imag
    return y


def quantize_f32_rows(x: np.ndarray):
    """float32 rows [..., D] -> (codes uint8, scales float32): scale = fl32(amax / 448),
    code = e4m3(fl32(x / scale)); an all-zero row gets scale 0 and codes 0."""
    amax = np.max(np.abs(x), axis=-1)
    scale = (amax / np.float32(448)).astype(np.float32)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.where(amax[..., None] > 0, x / scale[..., None], np.float32(0)).astype(np.float32)
    return e4m3_encode(q.reshape(-1)).reshape(x.shape), scale


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lens, sm_scale: float):
    """float64 [T, Hq, D] for T = sum(lens) packed tokens (inputs any float type), and two
    magnitudes per element or row: sum_j w_j |v_j| [T, Hq, D] and
    max_j sm_scale sum_d |q_d k_jd| [T, Hq, 1].  Values of unseen tokens are not touched."""
    q, k, v = (x.detach().cpu().double() for x in (q, k, v))
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, mag, dot = torch.zeros(T, Hq, D).double(), torch.zeros(T, Hq, D).double(), \
        torch.zeros(T, Hq, 1).double()
    a = 0
    for L in lens:
        b = a + int(L)
        for hq in range(Hq):
            K, V = k[a:b, hq // G], v[a:b, hq // G]
            for i0 in range(0, b - a, 512):
                i1 = min(b - a, i0 + 512)
                seen = torch.arange(i1)[None, :] <= torch.arange(i0, i1)[:, None]
                Q = q[a + i0:a + i1, hq]
                s = (sm_scale * Q @ K[:i1].T).masked_fill(~seen, -torch.inf)
                w = torch.softmax(s, dim=1)
                out[a + i0:a + i1, hq] = w @ V[:i1]
                mag[a + i0:a + i1, hq] = w @ V[:i1].abs()
                dot[a + i0:a + i1, hq, 0] = (sm_scale * Q.abs() @ K[:i1].abs().T) \
                    .masked_fill(~seen, 0).amax(dim=1)
        a = b
    return out, mag, dot
