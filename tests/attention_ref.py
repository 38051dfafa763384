"""Plain 64-bit references of the key-value cache and the attention operators (test
infrastructure; shares no code with the library).  CPU tensors and numpy arrays."""
from __future__ import annotations

import numpy as np
import torch

import oracle

BLOCK = {"mxfp8": 32, "nvfp4": 16, "mxfp4": 32}
RULE = {"ocp": oracle.MX_OCP_FLOOR, "ceil": oracle.MX_CEIL}


def encode_rows(fmt, x, tscale=None, rule="ocp"):
    """x fp32 [tokens, heads, dim] -> codes uint8 [tokens, heads, row], scales uint8 [tokens, heads, blocks]."""
    t, h, d = x.shape
    flat = np.ascontiguousarray(x.reshape(t * h, d), np.float32)
    if fmt == "mxfp4":
        codes, scales = oracle.mxfp4_quantize(flat, RULE[rule])
    elif fmt == "mxfp8":
        codes, scales = oracle.mxfp8_quantize(flat, RULE[rule])
    else:
        s = np.tile(np.asarray(tscale, np.float32), t)[:, None]
        blocks = flat.reshape(t * h, d // 16, 16)
        amax = np.abs(blocks).max(-1)
        with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
            q = (amax / (np.float32(6.0) * s)).astype(np.float32)
        q = np.where(amax == 0, np.float32(0), q)
        scales = oracle.e4m3_encode_array(q)
        values = np.array([oracle.e4m3_decode(int(b)) for b in range(256)], np.float32)
        step = (values[scales] * s).astype(np.float32)[..., None]
        with np.errstate(divide="ignore", invalid="ignore"):
            y = (blocks / step).astype(np.float32)
        y = np.where(step == 0, np.copysign(np.float32(0), blocks), y)
        n = oracle.e2m1_encode_array(y.reshape(-1)).reshape(t * h, d)
        codes = (n[:, 0::2] | (n[:, 1::2] << 4)).astype(np.uint8)
    return codes.reshape(t, h, -1), scales.reshape(t, h, -1)


def decode_rows(fmt, codes, scales, tscale=None):
    """The inverse in float64: [tokens, heads, dim]."""
    t, h, row = codes.shape
    c, s = codes.reshape(t * h, row), scales.reshape(t * h, -1)
    if fmt == "mxfp4":
        x = oracle.mxfp4_to_f64(c, s)
    elif fmt == "mxfp8":
        x = oracle.mxfp8_to_f64(c, s)
    else:
        x = oracle.nvfp4_to_f64(c, s, np.tile(np.asarray(tscale, np.float32), t), per_row=True)
    return np.asarray(x, np.float64).reshape(t, h, -1)


def attention(q, k, v, scale, first, last):
    """q [queries, heads, dim], k and v [keys, kv heads, dim] float64; query i sees keys first[i] ..
    last[i] - 1.  Returns out, lse, and the bound's terms: sum_j p_j |v_j| and, per row, the largest
    scale * sum |q| |k| over the keys it sees."""
    n, heads, dim = q.shape
    group = heads // k.shape[1]
    out, lse = torch.zeros(n, heads, dim, dtype=torch.float64), torch.full((n, heads), -float("inf"), dtype=torch.float64)
    mass, size = torch.zeros_like(out), torch.zeros(n, heads, dtype=torch.float64)
    for i in range(n):
        a, b = int(first[i]), int(last[i])
        if b <= a:
            continue
        for h in range(heads):
            kk, vv = k[a:b, h // group], v[a:b, h // group]
            z = (kk @ q[i, h]) * scale
            lse[i, h] = torch.logsumexp(z, 0)
            p = torch.exp(z - lse[i, h])
            out[i, h] = p @ vv
            mass[i, h] = p @ vv.abs()
            size[i, h] = ((kk.abs() @ q[i, h].abs()) * scale).max()
    return out, lse, mass, size


def check(got, lse_got, ref, dim, weight_ulp, what, v_abs_sum=None):
    """|out - ref| <= (u + 4 e) sum p|v| + the output's own rounding.

    u (`weight_ulp`): the softmax weights are rounded to 16 bits, relative error at most 2^-8 (bf16)
    or 2^-11 (f16).  e bounds a score's error, which moves numerator and denominator alike: `dim`
    fp32 additions and two products by the scale, (dim + 4) 2^-23 of scale * sum|q||k|, and 2^-19
    for exp2, log2 and the sums.  (f16 weights below 2^-14 carry an absolute error of 2^-25: `v_abs_sum`.)"""
    out, lse, mass, size = ref
    assert tuple(got.shape) == tuple(out.shape), what
    e = (dim + 4) * 2.0 ** -23 * size + 2.0 ** -19
    lim = (weight_ulp + 4 * e[..., None]) * mass
    if v_abs_sum is not None:
        lim = lim + 2.0 ** -24 * v_abs_sum
    if got.dtype == torch.bfloat16:
        lim = lim * (1 + 2.0 ** -8) + 2.0 ** -8 * out.abs()
    g = got.detach().cpu().double()
    assert bool(torch.isfinite(g).all()), f"{what}: non-finite outputs"
    err = (g - out).abs()
    bad = err > lim + 1e-30
    assert not bool(bad.any()), f"{what}: {int(bad.sum())} of {bad.numel()} out of bound, first {bad.nonzero()[0].tolist()}, worst {float((err / (lim + 1e-30)).max()):.3g}"
    if lse_got is not None:
        x = lse_got.detach().cpu().double()
        empty = torch.isinf(lse)
        assert bool((x[empty] == -float("inf")).all()), what
        d = (x - lse).abs()[~empty]
        lim = (2 * e + 2.0 ** -20 * lse.abs().clamp(max=1e30))[~empty]
        assert bool((d <= lim).all()), f"{what}: lse off by {float(d.max()):.3g}"
