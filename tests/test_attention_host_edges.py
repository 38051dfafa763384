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


def test_workspace_sizes_are_kept_by_device(fp4, monkeypatch):  # noqa: F811
    """The library sizes a workspace by the current device's CUs: what one device needs says nothing of another."""
    class Lib:  # the two queries on devices of 256 and 304 CUs
        attn_prefill_workspace = staticmethod(lambda *a: cus[now] * 16)
        attn_decode_paged_workspace = staticmethod(lambda *a: cus[now] * 32)

    cus, now = {0: 256, 1: 304}, 0
    monkeypatch.setattr(fp4, "lib", lambda: Lib)
    monkeypatch.setattr(torch.cuda, "is_initialized", lambda: True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now)
    cache = type("Sizes", (), dict(kv_heads=2, page_size=16, head_dim=64, device="cpu"))
    fp4._decode_need.cache_clear(), fp4._prefill_need.cache_clear()
    for now in (0, 1, 0):
        assert fp4.attn_prefill_workspace(5, 8, 90001, 2, 64, 1, device="cpu").numel() == cus[now] * 16
        assert fp4.attn_decode_paged_workspace(cache, 3, 8, 12345).numel() == cus[now] * 32
    fp4._decode_need.cache_clear(), fp4._prefill_need.cache_clear()


def test_short_prompts_are_not_split(fp4):  # noqa: F811
    """The keys of a row are its sequence's, not the batch's: many short prompts need no partial results."""
    need = fp4.lib().attn_prefill_workspace
    assert need(1024, 8, 1024, 2, 128, 16) == 0      # 16 prompts of 64 tokens
    assert need(3200, 4, 3200, 1, 128, 16) == 0      # 16 of 200
    assert need(16, 8, 16 * 40000, 2, 128, 16) > 0   # 16 queries, each behind 39999 keys
    assert need(16, 8, 60000, 2, 128, 16) > 0        # one of them may have nearly all the keys
