"""The paged cache's operators at the ends of their ranges."""
import numpy as np
import pytest
import torch

import long_context_decode_nuq_b200 as K
import paged_testlib as R
from long_context_decode_nuq_b200.paged import PagedSession

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------ quantizer
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("exp", [-64, -39, -38, -37, -10, -9, -8, 0, 38, 64])
def test_append_values_far_past_the_largest_scale(dtype, exp):
    """The type's extremes and infinities of both signs, beside values of every size: a value past
    6 * 448 * 2^exp is stored as that, with its own sign."""
    big = float(torch.finfo(DT[dtype]).max)
    x = torch.randn((64, 1, 128), generator=torch.Generator().manual_seed(1)).to(DT[dtype])
    sizes = torch.exp2(torch.linspace(-100, 127, 64) if dtype == "bf16" else torch.linspace(-14, 14, 64))
    x[:, 0, :32] = (x[:, 0, :32].float() * sizes[:, None]).clamp(-big, big).to(DT[dtype])
    for j, (a, b) in enumerate([(big, -big), (float("inf"), -float("inf")), (-float("inf"), -big), (big, float("nan")), (-big / 2, 1.0)]):
        x[j::5, 0, 32 + 16 * j], x[j::5, 0, 37 + 16 * j] = a, b
    x[::7, 0, 112:] = -big
    want = torch.tensor(R.quantize(x.double().numpy(), exp) * 2.0 ** -exp).to(DT[dtype])
    c = K.PagedCache(K.make_paged_cfg(1, 1, 128, 16, 4, 4, DT[dtype], exp, exp))
    x, slots = x.cuda(), i32(range(64))
    K.kvq_paged_append(c, x, x, slots)
    kh, vh = torch.empty_like(x), torch.empty_like(x)
    # read with exponent 0, code * scale: exact in both types
    K.kvq_paged_dequantize(K.PagedCache(K.make_paged_cfg(1, 1, 128, 16, 4, 4, DT[dtype]), pool=c.pool), slots, kh, vh)
    assert torch.equal(kh.cpu(), want) and torch.equal(vh.cpu(), want)
    assert K.kvq_paged_get_status(c) == 0


# ------------------------------------------------------------------------------ pages
@pytest.mark.parametrize("P", [16, 128])
@pytest.mark.parametrize("B,width", [(3, 9), (40, 60), (1500, 5)])
def test_release_of_tables_whose_first_pages_are_gone(P, B, width):
    """Pages behind a window that were given back early have entries of -1: release leaves those
    out, and every page is on the list exactly once."""
    r = np.random.RandomState(B)
    lens = r.randint(0, width * P + 1, B)
    need = -(-lens // P)
    pages = int(need.sum()) + 3
    c = K.PagedCache(K.make_paged_cfg(1, 1, 64, P, pages, width, torch.bfloat16))
    perm, table, at = r.permutation(pages), np.full((B, width), -1), 0
    early, late, ended = [], [], r.rand(B) < 0.7
    ended[0] = True
    for b in range(B):
        own, gone = perm[at:at + need[b]], r.randint(0, need[b] + 1)
        at += need[b]
        table[b, gone:need[b]] = own[gone:]
        early += own[:gone].tolist()
        if ended[b]:
            late += own[gone:].tolist()
    first = perm[at:].tolist() + early  # the list while the requests run
    free = np.full(pages, -9)
    free[:len(first)] = first
    d_lens, d_table, d_free, n_free = i32(lens), i32(table), i32(free), i32([len(first)])
    K.kvq_page_release(c, d_lens, i32(ended), d_table, d_free, n_free)
    assert K.kvq_paged_get_status(c) == 0
    assert d_free.tolist()[:int(n_free)] == first + late
    assert d_lens.tolist() == np.where(ended, 0, lens).tolist()
    assert np.array_equal(d_table.cpu().numpy(), np.where(ended[:, None], -1, table))
    # what the plan hands out next is a page
    n_new = i32([0] * (B - 1) + [P]) if ended[-1] else i32([P] + [0] * (B - 1))
    slots, pos = i32([0] * P), i32([0] * P)
    if int(n_free):
        K.kvq_page_plan(c, d_lens, n_new, d_table, d_free, n_free, i32([0] * (B + 1)), d_lens, n_free, slots, pos)
        assert K.kvq_paged_get_status(c) == 0 and bool((slots >= 0).all())


def test_release_reports_entries_outside_the_pool():
    c = K.PagedCache(K.make_paged_cfg(1, 1, 64, 16, 6, 4, torch.bfloat16))
    lens, table, free, n_free = i32([64, 33]), i32([[2, 6, -1, 0], [-1, 4, 5, -1]]), i32([1, 0, 0, 0, 0, 0]), i32([1])
    K.kvq_page_release(c, lens, i32([0, 1]), table, free, n_free)
    assert free.tolist()[:3] == [1, 4, 5] and int(n_free) == 3 and K.kvq_paged_get_status(c) == 0
    K.kvq_page_release(c, lens, i32([1, 1]), table, free, n_free)
    assert free.tolist()[:5] == [1, 4, 5, 2, 0] and int(n_free) == 5 and K.kvq_paged_get_status(c) == K.KVQ_STATUS_BAD_PAGE
    assert bool((table == -1).all()) and not lens.any()


def test_plan_reads_no_further_than_its_list():
    """A list of fewer entries than n_free says (here with more memory behind it, which names other
    pages): what counts is the list."""
    c = K.PagedCache(K.make_paged_cfg(1, 1, 64, 16, 20, 4, torch.bfloat16))
    memory = i32([7, 8, 9, 0, 1, 2, 3, 4, 5, 6])
    lens, new, table, n_free = i32([0, 0, 0]), i32([20, 33, 16]), i32(np.full((3, 4), -1)), i32([10])
    slots, pos = i32([0] * 69), i32([0] * 69)
    K.kvq_page_plan(c, lens, new, table, memory[:3], n_free, i32([0] * 4), lens, n_free, slots, pos)
    # three pages: the first takes two, the second lacks three
    assert table.tolist() == [[9, 8, -1, -1], [-1] * 4, [-1] * 4]
    assert lens.tolist() == [20, 0, 0] and n_free.tolist() == [1]
    assert slots.tolist() == list(range(144, 160)) + list(range(128, 132)) + [-1] * 49
    assert K.kvq_paged_get_status(c) == K.KVQ_STATUS_NO_PAGES


# ------------------------------------------------------------------------------ attention
@pytest.mark.parametrize("B,Hkv,n,T,splits", [(1, 1, 1, 1 << 26, 1), (1, 1, 16, 1 << 26, 1), (5, 64, 1, 1 << 25, 0), (1, 1, 20, 1 << 26, 1), (1, 1, 1, 1 << 26, 0)])
def test_attention_sums_do_not_drift(B, Hkv, n, T, splits):
    """Equal weights over values of one sign, the same few pages again and again, so that the sums
    only grow.  Tolerance: the output's half step, and 2^13 times in a row at most that a sum is cut
    off, by less than a step (2^-23) of what has been summed by then: 2^13 / 2 * 2^-23 = 2^-11 of
    the whole.  (Chunks: 2^17 tokens, 16 at a time.  Few rows: 2^15 tokens a warp, 16 at a time,
    where an instruction may cut off up to four times.)  Parts are joined in binary32: 2^-24 for
    each of up to 2^10, as the warps and blocks that join them add theirs in a tree."""
    P, D, pages = 128, 64, 64
    c = K.PagedCache(K.make_paged_cfg(Hkv, Hkv, D, P, pages, T // P, torch.float16))
    v = torch.rand((pages * P, Hkv, D), generator=torch.Generator("cuda").manual_seed(1), device="cuda").half() + 0.5
    slots = torch.arange(pages * P, dtype=torch.int32, device="cuda")
    K.kvq_paged_append(c, torch.zeros_like(v), v, slots)
    kh = torch.empty_like(v)
    K.kvq_paged_dequantize(c, slots, kh, v)
    want = v.double().mean(0)
    table = (torch.arange(T // P, device="cuda") % pages).int().repeat(B, 1)
    q = torch.randn((B * n, Hkv, D), device="cuda").half()
    out = torch.empty_like(q)
    ws = torch.empty(max(16, K.kvq_paged_attention_workspace(c.cfg, B, B * n, n, T, splits)), dtype=torch.uint8, device="cuda")
    K.kvq_paged_attention(c, q, i32(range(0, B * n + 1, n)), i32([T] * B), table, n, T, 1.0, out, ws, splits=splits)
    # the last query sees every page equally often
    worst = ((out[n - 1::n].double() - want).abs() / want).max().item()
    assert worst <= 2.0 ** -11 * 1.01 + 2.0 ** -11 + 2.0 ** -14, worst
    assert K.kvq_paged_get_status(c) == 0


# ------------------------------------------------------------------------------ together
def test_session_steps_without_tokens():
    cfg = K.make_paged_cfg(4, 2, 64, 16, 40, 20, torch.bfloat16)
    rope = K.make_rope_cfg(4, 2, 64, 64, [0] * 32, torch.bfloat16)
    freqs = 1e4 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    s = PagedSession(cfg, 1, 2, rope, freqs)
    for new in ([0, 0], [5, 0], [0, 0], [1, 1]):
        n = sum(new)
        q, k, v = (torch.randn((n, h, 64), device="cuda").bfloat16() for h in (4, 2, 2))
        out = torch.full_like(q, float("nan"))
        s.begin(i32(new), n, max(new))
        s.attend(0, q, k, v, 0.125, out)
        assert bool(torch.isfinite(out.float()).all())
    assert s.lens.tolist() == [6, 1] and s.status() == 0


def test_rope_cfg_filled_by_hand():
    x = torch.randn((5, 2, 64), device="cuda")
    pos, freqs = i32([np.arange(5), np.arange(5) * 3]), torch.rand(16, dtype=torch.float64, device="cuda")
    a = K.make_rope_cfg(2, 0, 64, 32, [0, 1] * 8, torch.float32)
    b = K.RopeCfg(2, 0, 64, 32, 2, 0, 2, a.pair_axis)
    outs = [torch.zeros_like(x) for _ in range(2)]
    for cfg, out in zip((a, b), outs):
        K.kvq_rope(cfg, x, None, pos, freqs, out, None)
    assert torch.equal(*outs) and not torch.equal(outs[0], x)
