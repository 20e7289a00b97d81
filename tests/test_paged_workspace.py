"""Workspace sizes of kvq_paged_attention: bounded, and one for the largest step serves the others."""
import random

import pytest
import torch

import long_context_decode_nuq_b200 as K


def cfg(Hq=32, Hkv=8, D=128, P=64, width=1 << 20):
    return K.make_paged_cfg(Hq, Hkv, D, P, 1000, width, torch.bfloat16)


@pytest.mark.parametrize("B,n,T", [(1, 1184, 32768), (1, 2048, 32768), (1, 10688, 131072), (64, 2048, 131072), (3, 40, 100000), (1, 17, 131072)])
def test_workspace_is_bounded(B, n, T):
    """With the library's choice, at most six waves of split row blocks (256 rows each) on 148 SMs,
    whatever the number of queries, and no more than one part per 128 tokens of every row."""
    for total in (n, B * n):
        rows = min(6 * 148 * 256, total * 32 * -(-T // 128))
        assert K.kvq_paged_attention_workspace(cfg(), B, total, n, T) <= max(rows * 130 * 4, 296 * 2 * 16 * 130 * 4 + B * 8 * 16)


def test_workspace_over_the_longest_split():
    """Past 2^17 tokens every row has a part for each 2^17 of them."""
    n = [K.kvq_paged_attention_workspace(cfg(), 1, 20000, 20000, T) for T in (1 << 17, (1 << 17) + 1, 1 << 20)]
    assert n[0] <= 6 * 148 * 256 * 130 * 4 and n[1:] == [p * 20000 * 32 * 130 * 4 for p in (2, 8)]


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 128), (8, 8, 64), (64, 1, 128), (7, 1, 64), (32, 2, 128)])
def test_workspace_for_the_largest_serves_smaller(Hq, Hkv, D):
    r = random.Random(Hq)
    log = lambda lo, hi: max(lo, min(hi, int(lo * (hi / lo) ** r.random())))  # noqa: E731
    c = cfg(Hq, Hkv, D)
    for _ in range(3000):
        B, q, T = log(1, 400), log(1, 5000), log(1, 1 << 21)
        total = log(1, B * q)
        b = [r.choice((x, log(1, x))) for x in (B, total, q, T)]
        assert K.kvq_paged_attention_workspace(c, *b) <= K.kvq_paged_attention_workspace(c, B, total, q, T), (B, total, q, T, b)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,window", [(32, 8, 128, 0), (24, 3, 64, 0), (32, 8, 128, 700), (64, 2, 64, 3000)])
def test_one_workspace_for_steps_of_every_size(Hq, Hkv, D, window):
    """Each call within the same workspace gives the bits of a call with one of its own, and nothing
    past its end is written.  (Row blocks whole, some split, all split; a window that changes the plan.)"""
    P, T, pages = 64, 9000, 300
    c = K.PagedCache(K.make_paged_cfg(Hq, Hkv, D, P, pages, T // P + 1, torch.bfloat16))
    g = torch.Generator("cuda").manual_seed(1)
    kv = torch.randn((pages * P, Hkv, D), generator=g, device="cuda").bfloat16()
    K.kvq_paged_append(c, kv, kv, torch.arange(pages * P, dtype=torch.int32, device="cuda"))
    top = K.kvq_paged_attention_workspace(c.cfg, 40, 8000, 2500, T)
    shared = torch.full((top + 4096,), 0xAB, dtype=torch.uint8, device="cuda")
    for B, n, t in ((1, 2500, 9000), (1, 1200, 9000), (2, 90, 8192), (40, 200, 700), (40, 3, 300), (3, 1, 9000), (7, 333, 2000), (16, 40, 5000)):
        assert K.kvq_paged_attention_workspace(c.cfg, B, B * n, n, t) <= top
        table = torch.stack([torch.randperm(pages, generator=g, device="cuda")[:T // P + 1] for _ in range(B)]).int()
        lens = torch.tensor([t - b * 5 for b in range(B)], dtype=torch.int32, device="cuda")
        cu = torch.arange(0, B * n + 1, n, dtype=torch.int32, device="cuda")
        q = torch.randn((B * n, Hq, D), generator=g, device="cuda").bfloat16()
        own = torch.full((K.kvq_paged_attention_workspace(c.cfg, B, B * n, n, t),), 0xFF, dtype=torch.uint8, device="cuda")
        outs = []
        for ws in (own, shared[:top]):
            out, lse = torch.full_like(q, 7.0), torch.full((B * n, Hq), 7.0, device="cuda")
            K.kvq_paged_attention(c, q, cu, lens, table, n, t, D ** -0.5, out, ws, window=window, lse=lse)
            outs.append((out, lse))
        assert torch.equal(*(x.view(torch.int16) for x, _ in outs)) and torch.equal(*(x for _, x in outs))
        assert bool(torch.isfinite(outs[0][0].float()).all()) and bool((shared[top:] == 0xAB).all())
        # all splits' parts joined: the same within what a split moves, against one part per row
        one = torch.empty(max(16, K.kvq_paged_attention_workspace(c.cfg, B, B * n, n, t, 1)), dtype=torch.uint8, device="cuda")
        ref = torch.empty_like(q)
        K.kvq_paged_attention(c, q, cu, lens, table, n, t, D ** -0.5, ref, one, window=window, splits=1)
        # a rounding of each output, 2^-8, and P's 2^-11 of a value of at most 6 times 1
        assert bool(((outs[0][0].float() - ref.float()).abs() <= ref.float().abs() * 2.0 ** -7 + 2 * 6 * 2.0 ** -11).all())
    assert K.kvq_paged_get_status(c) == 0
