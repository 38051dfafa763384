"""Attention at the edges: sequences that end inside a tile before rows that are not numbers, values
that are not numbers in masked places, scores of any size, weights far below the largest one,
single-token buffers of any stride, and every part of the launch rules."""
import numpy as np
import pytest
import torch

import attention_ref as ref

pytestmark = pytest.mark.gpu


def _fp4():
    import block_scaled_fp4_04_amd as fp4

    return fp4


def _cu(lens):
    return torch.tensor(np.cumsum([0] + list(lens)), dtype=torch.int32, device="cuda")


def _randn(g, *shape):
    return torch.randn(*shape, generator=g).to(torch.bfloat16)


@pytest.mark.parametrize("dim", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_prompt_ends_before_nan(dim, causal):
    """Every second sequence's keys and values are NaN, and so is the memory behind the last one: rows of a
    tile past a sequence's end count as zeros wherever the end falls within the tile."""
    fp4 = _fp4()
    g = torch.Generator().manual_seed(dim)
    ends = [1, 5, 7, 8, 9, 15, 16, 17, 20, 24, 31, 32, 33, 40, 48, 63, 65, 1]
    lens = [n for e in ends for n in (e, 3)][:-1]
    n, heads, kv = sum(lens), 2, 1
    q, k, v = _randn(g, n, heads, dim), _randn(g, n + 70, kv, dim), _randn(g, n + 70, kv, dim)
    offs = np.cumsum([0] + lens)
    for b in range(1, len(lens), 2):
        k[offs[b]:offs[b + 1]] = v[offs[b]:offs[b + 1]] = float("nan")
    k[n:] = v[n:] = float("nan")
    lse = torch.empty(n, heads, device="cuda")
    out = fp4.attn_prefill(q.cuda(), k.cuda()[:n], v.cuda()[:n], _cu(lens), _cu(lens), causal=causal, dtype=torch.float32, lse=lse)
    for b in range(0, len(lens), 2):
        at = slice(offs[b], offs[b + 1])
        m = lens[b]
        last = [i + 1 if causal else m for i in range(m)]
        want = ref.attention(q[at].double(), k[at].double(), v[at].double(), dim ** -0.5, [0] * m, last)
        ref.check(out[at], lse[at], want, dim, 2.0 ** -8, f"{m} keys before NaN, head_dim {dim}")
