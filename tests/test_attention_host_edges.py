"""Attention entry points on the host (nothing is launched): strides that are never followed, limits of
a launch, workspace sizes by device."""
import pytest
import torch

import test_attention_host as host
from test_attention_host import GPU, NO_DEVICE, fp4  # noqa: F401  (the fixture)


@pytest.mark.parametrize("room", [2, 32768, 1 << 20])
def test_one_token_of_a_head_major_buffer(fp4, room):  # noqa: F811
    """One key or query in a [heads, room, dim] buffer: its token stride is never followed, whatever the buffer's size."""
    buf = torch.empty(8, room, 128, dtype=torch.bfloat16, device="meta")
    for n in (1, 2):
        t = buf[:, :n].transpose(0, 1)
        tokens, heads, dim, tok, head = fp4._heads(t, fp4._BF16, "k")
        assert (tokens, heads, dim, head) == (n, 8, 128, room * 128)
        if not GPU:
            got = host._prefill(fp4, kn=n, heads=8, kv=8, dim=128, kt=tok, kh=head, vt=tok, vh=head, qn=n, qt=tok, qh=head,
                                ott=tok, oh=head)
            assert got == NO_DEVICE, n
