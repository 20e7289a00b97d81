"""The paged 4-bit cache against plain 64-bit forms: quantizer, page plan, attention, and all of
them as a serving loop uses them."""
import random

import numpy as np
import pytest
import torch

import long_context_decode_nuq_b200 as K
import paged_testlib as R
from long_context_decode_nuq_b200.paged import PagedSession

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


def make(dtype="bf16", Hq=8, Hkv=2, D=128, P=16, pages=64, width=16, ke=0, ve=0):
    cfg = K.make_paged_cfg(Hq, Hkv, D, P, pages, width, DT[dtype], ke, ve)
    c = K.PagedCache(cfg)
    c.pool.fill_(0xFF)  # NaN scales wherever nothing is written
    return c


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def rand(shape, dtype, seed, strong=False):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    if strong:
        x[..., ::21] *= 6.0
    return x.to(DT[dtype])


def f64(t):
    return t.double().cpu().numpy()


# ------------------------------------------------------------------------------ quantizer
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P,Hkv,n,ke,ve", [(16, 1, 1, 0, 0), (32, 3, 77, 0, 0), (128, 8, 300, 3, -5), (64, 2, 130, -64, 64)])
def test_append_stores_nearest_values(dtype, D, P, Hkv, n, ke, ve):
    pages = -(-n // P) + 2
    c = make(dtype, Hkv, Hkv, D, P, pages, pages, ke, ve)
    # rows of a wider projection: heads contiguous, tokens apart; sizes from tiny to the largest
    wide = rand((n, 2 * Hkv + 1, D), dtype, 3, True) * torch.exp2(torch.randint(-12, 12, (n, 2 * Hkv + 1, 1), device="cuda").float()).to(DT[dtype])
    k, v = wide[:, :Hkv], wide[:, Hkv + 1:]
    slots = torch.randperm(pages * P, device="cuda")[:n].int()
    K.kvq_paged_append(c, k, v, slots)
    kh, vh = torch.empty_like(k, memory_format=torch.contiguous_format), torch.empty((n, Hkv, D), dtype=DT[dtype], device="cuda")
    K.kvq_paged_dequantize(c, slots, kh, vh)
    big = float(torch.finfo(DT[dtype]).max)
    for got, x, e in ((kh, k, ke), (vh, v, ve)):
        want = torch.tensor(np.clip(R.quantize(f64(x), e), -big, big)).to(DT[dtype])
        assert torch.equal(got.cpu(), want)
    assert K.kvq_paged_get_status(c) == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_append_every_finite_value_and_ties(dtype):
    """Every finite 16-bit number, beside each of the values that set its group's scale."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    x = bits.view(DT[dtype])
    x = x[torch.isfinite(x.float())]
    for top in (6.0, 5.5, 448.0 * 6, 0.013, 7.0, 60000.0):
        g = torch.full((-(-x.numel() // 15), 16), top).to(DT[dtype])
        small = torch.where(x.float().abs() <= top, x, torch.zeros_like(x))
        g[:, :15] = torch.nn.functional.pad(small, (0, g.shape[0] * 15 - x.numel())).view(-1, 15)
        g = torch.nn.functional.pad(g, (0, 0, 0, -g.shape[0] % 8)).view(-1, 1, 128).cuda()
        n = g.shape[0]
        c = make(dtype, 1, 1, 128, 16, -(-n // 16), 1)
        slots = torch.arange(n, device="cuda").int()
        K.kvq_paged_append(c, g, g, slots)
        kh, vh = torch.empty_like(g), torch.empty_like(g)
        K.kvq_paged_dequantize(c, slots, kh, vh)
        big = float(torch.finfo(DT[dtype]).max)
        want = torch.tensor(np.clip(R.quantize(f64(g)), -big, big)).to(DT[dtype])
        assert torch.equal(kh.cpu(), want) and torch.equal(vh.cpu(), want)


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_append_special_values(dtype):
    x = rand((4, 1, 64), dtype, 1)
    x[0, 0, 3] = float("nan")
    x[1, 0, :16] = float("nan")
    x[1, 0, 20] = float("-inf")
    x[2, 0, 40], x[2, 0, 41] = float("inf"), float("nan")
    x[3] = 0
    c = make(dtype, 1, 1, 64, 16, 1, 1)
    slots = i32(range(4))
    K.kvq_paged_append(c, x, x, slots)
    kh, vh = torch.empty_like(x), torch.empty_like(x)
    K.kvq_paged_dequantize(c, slots, kh, vh)
    want = torch.tensor(R.quantize(f64(x))).to(DT[dtype])
    assert torch.equal(kh.cpu(), want) and torch.equal(vh.cpu(), want)
    assert f64(kh)[1, 0, 20] == -2688 and f64(kh)[2, 0, 40] == 2688


def test_append_skips_and_reports_slots():
    c = make(pages=2)
    k = rand((5, 2, 128), "bf16", 1)
    before = c.pool.clone()
    K.kvq_paged_append(c, k, k, i32([-1] * 5))
    assert torch.equal(c.pool, before) and K.kvq_paged_get_status(c) == 0
    K.kvq_paged_append(c, k, k, i32([32, -2, 2**31 - 1, -2**31, -1]))
    assert torch.equal(c.pool, before) and K.kvq_paged_get_status(c) == K.KVQ_STATUS_BAD_PAGE
    K.kvq_paged_reset(c)
    kh, vh = torch.ones_like(k), torch.ones_like(k)
    K.kvq_paged_dequantize(c, i32([-1, 32, -1, -9, -1]), kh, vh)
    assert not kh.any() and not vh.any() and K.kvq_paged_get_status(c) == K.KVQ_STATUS_BAD_PAGE
    K.kvq_paged_append(c, k[:0], k[:0], i32([]))
    torch.cuda.synchronize()


def test_append_leaves_other_tokens_alone():
    c = make(pages=3, P=32)
    a, b = rand((96, 2, 128), "bf16", 1), rand((1, 2, 128), "bf16", 2)
    K.kvq_paged_append(c, a, a, i32(range(96)))
    K.kvq_paged_append(c, b, b, i32([41]))
    kh, vh = torch.empty_like(a), torch.empty_like(a)
    K.kvq_paged_dequantize(c, i32(range(96)), kh, vh)
    want = R.quantize(f64(a))
    want[41] = R.quantize(f64(b))[0]
    assert np.array_equal(f64(kh), want) and np.array_equal(f64(vh), want)


# ------------------------------------------------------------------------------ page plan
def run_plan(c, lens, n_new, table, free, n_free, capacity, in_place=False):
    B = len(lens)
    L, N = i32(lens), i32(n_new)
    cu, nf = torch.empty(B + 1, dtype=torch.int32, device="cuda"), i32([n_free])
    lo, no = (L, nf) if in_place else (torch.empty_like(L), torch.empty_like(nf))
    slots, pos = torch.full((capacity,), -7, dtype=torch.int32, device="cuda"), torch.full((capacity,), -7, dtype=torch.int32, device="cuda")
    K.kvq_page_plan(c, L, N, table, free, nf, cu, lo, no, slots, pos)
    return [x.cpu().numpy() for x in (cu, lo, slots, pos, no)]


@pytest.mark.parametrize("P", [16, 128])
@pytest.mark.parametrize("B,T,n,width,spare,extra", [
    (1, 0, 1, 4, 5, 0), (1, 100, 0, 8, 0, 3), (5, 60, 9, 8, 50, 0), (33, 300, 40, 20, 7, 5), (33, 300, 40, 20, 7, -300),
    (1024, 90, 3, 8, 4000, 0), (1025, 90, 5, 8, 300, 9), (3000, 500, 20, 40, 9000, 100), (9001, 100, 6, 9, 20000, 3), (2, 9000, 20000, 2000, 3000, 0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_plan(P, B, T, n, width, spare, extra, in_place):
    r = random.Random(B * 31 + P)
    lens = [min(r.randrange(T + 1), width * P) for _ in range(B)]
    new = [r.choice([0, 1, r.randrange(n + 1)]) for _ in range(B)]
    have = [-(-a // P) for a in lens]
    perm = np.random.RandomState(B).permutation(sum(have) + spare + 1).astype(np.int32)
    pages = len(perm)
    c = make(pages=pages, P=P, width=width, Hq=1, Hkv=1, D=64)
    table = np.full((B, width), -5, np.int32)
    at = 0
    for b, m in enumerate(have):
        table[b, :m] = perm[at:at + m]
        at += m
    free = np.concatenate([perm[at:], np.zeros(pages - spare - 1, np.int32)])[:pages]
    capacity = max(sum(new) + extra, 0)
    d_table = i32(table)
    got = run_plan(c, lens, new, d_table, i32(free), spare + 1, capacity, in_place)
    cu, out, slots, pos, left, status = R.plan(lens, new, table, free, spare + 1, P, width, capacity)
    for g, w, name in zip(got, (cu, out, slots, pos, [left]), ("cu", "len", "slots", "pos", "n_free")):
        assert np.array_equal(g, np.asarray(w)), name
    assert np.array_equal(d_table.cpu().numpy(), table)
    assert K.kvq_paged_get_status(c) == status


def test_plan_and_release_cycle():
    """Requests that come and go never share a page, and every page comes back."""
    P, pages, width, B = 16, 60, 12, 9
    c = make(pages=pages, P=P, width=width, Hq=1, Hkv=1, D=64)
    free, n_free = i32(np.random.RandomState(0).permutation(pages)), i32([pages])
    lens, table = i32([0] * B), i32(np.full((B, width), -1))
    cu = torch.empty(B + 1, dtype=torch.int32, device="cuda")
    r = random.Random(2)
    for step in range(40):
        new = [r.choice([0, 1, 1, r.randrange(70)]) for _ in range(B)]
        slots = torch.empty(sum(new) + 1, dtype=torch.int32, device="cuda")
        K.kvq_page_plan(c, lens, i32(new), table, free, n_free, cu, lens, n_free, slots, torch.empty_like(slots))
        K.kvq_page_release(c, lens, i32([r.random() < 0.15 for _ in range(B)]), table, free, n_free)
        ln, tb, nf = lens.cpu().numpy(), table.cpu().numpy(), int(n_free)
        held = [int(x) for b in range(B) for x in tb[b, :-(-int(ln[b]) // P)]]
        assert sorted(held + free.cpu().numpy()[:nf].tolist()) == list(range(pages))
    assert K.kvq_paged_get_status(c) & ~(K.KVQ_STATUS_NO_PAGES | K.KVQ_STATUS_LEN_OVERFLOW) == 0
    K.kvq_page_release(c, lens, i32([1] * B), table, free, n_free)
    assert int(n_free) == pages and not lens.any() and bool((table == -1).all())


def test_release_more_than_fits_is_reported():
    c = make(pages=4, width=4, Hq=1, Hkv=1, D=64)
    lens, table, free, n_free = i32([64]), i32([[0, 1, 2, 3]]), i32([9, 9, 9, -3]), i32([3])
    K.kvq_page_release(c, lens, i32([1]), table, free, n_free)
    assert free.tolist() == [9, 9, 9, 0] and int(n_free) == 4
    assert K.kvq_paged_get_status(c) == K.KVQ_STATUS_BAD_PAGE


# ------------------------------------------------------------------------------ attention
def fill(c, dtype, lens, seed, shuffle=True):
    """Tokens of each request, quantized into scattered pages: the table and the stored values."""
    P, cfg = c.cfg.page_tokens, c.cfg
    need = [-(-a // P) for a in lens]
    perm = np.random.RandomState(seed).permutation(cfg.num_pages)
    table = np.full((len(lens), cfg.max_pages), -1, np.int32)
    at, kv = 0, []
    for b, a in enumerate(lens):
        table[b, :need[b]] = perm[at:at + need[b]]
        at += need[b]
        k, v = rand((a, cfg.Hkv, cfg.D), dtype, seed + 2 * b, True), rand((a, cfg.Hkv, cfg.D), dtype, seed + 2 * b + 1) + 0.3
        t = np.arange(a)
        K.kvq_paged_append(c, k, v, i32(table[b, t // P] * P + t % P))
        kv.append((R.quantize(f64(k), cfg.k_exp), R.quantize(f64(v), cfg.v_exp)))
    return i32(table), kv


def check(got, lse, q, kv, news, scale, window, dtype):
    """Tolerance: the output's own rounding; P's rounding to fp16 (2^-11 of each term) and the
    exponential's 2^-22; a score's binary32 sums (D 2^-24 of sum |q k|, twice for truncation in the
    tensor cores, and the scaling's 2^-23 of it) move every weight by a factor e^d.  Below the normal
    numbers the steps are absolute: a weight is held as fp16 with its row's largest at 2^12 or more,
    so it is off by at most 2^-25 / 2^12 = 2^-37 of the largest, which is at most 1; an fp16 output
    by 2^-25.  (A query of 1000 gives weights of 1e-22 to all tokens but one: they are stored as 0.)"""
    at = 0
    for (k, v), n in zip(kv, news):
        o, l, pv, qk = R.attention(q[at:at + n], k, v, n, scale, window)
        d = qk * (q.shape[2] * 2.0 ** -23 + 2.0 ** -22) + 2.0 ** -20
        tol = np.abs(o) * float(torch.finfo(DT[dtype]).eps) / 2 * 1.01 + pv * (2.0 ** -11 + 2 * d[..., None])
        tol += len(k) * 2.0 ** -37 * np.abs(v).max(initial=0) + (2.0 ** -25 if dtype == "fp16" else 0)
        worst = (np.abs(f64(got[at:at + n]) - o) - tol).max(initial=-1)
        assert worst <= 0, worst
        if lse is not None:
            gl = f64(lse[at:at + n])
            empty = np.isinf(l)
            assert np.array_equal(np.isneginf(gl), empty)
            gl, l, d = gl[~empty], l[~empty], d[~empty]
            assert np.all(np.abs(gl - l) <= d + 2.0 ** -22 * (np.abs(l) + 20))
        at += n


CASES = [
    # dtype, D, P, Hkv, G, lens, new tokens, window, splits
    ("bf16", 128, 16, 1, 1, [1], [1], 0, 0),
    ("fp16", 128, 16, 2, 4, [0, 1, 15, 16, 17, 33], [1] * 6, 0, 0),
    ("bf16", 64, 32, 3, 1, [31, 32, 33, 64, 65, 700], [1] * 6, 0, 0),
    ("fp16", 64, 64, 1, 8, [1000, 3, 0, 129], [1] * 4, 0, 3),
    ("bf16", 128, 128, 2, 7, [517, 128, 127, 1], [1] * 4, 0, 1),
    ("bf16", 128, 16, 1, 16, [260, 31, 5], [1] * 3, 0, 7),
    ("fp16", 128, 32, 1, 64, [90, 300], [1, 1], 0, 0),
    ("bf16", 128, 16, 2, 4, [5000], [1], 0, 0),
    ("bf16", 128, 16, 2, 4, [5000], [1], 0, 256),
    ("bf16", 128, 32, 2, 4, [300, 40, 5, 0], [4, 4, 4, 0], 0, 0),
    ("fp16", 128, 64, 2, 4, [300, 40, 7], [7, 3, 7], 0, 2),
    ("bf16", 64, 16, 1, 3, [200, 33, 9], [11, 1, 5], 0, 0),
    ("bf16", 128, 16, 2, 1, [64, 300, 17], [40, 130, 17], 0, 0),
    ("fp16", 64, 128, 1, 5, [257, 80], [61, 80], 0, 4),
    ("fp16", 128, 16, 1, 4, [400, 150, 333], [150, 150, 77], 0, 0),
    # more queries than tokens: the first see nothing
    ("bf16", 128, 16, 1, 2, [3, 0, 20], [9, 5, 9], 0, 0),
    ("bf16", 128, 16, 1, 4, [3, 0, 60], [140, 33, 129], 0, 0),
    # windows: one token, odd, longer than the request
    ("bf16", 128, 16, 2, 4, [500, 77, 3], [1, 1, 1], 1, 0),
    ("fp16", 128, 32, 1, 8, [500, 77, 3], [1, 1, 1], 45, 2),
    ("bf16", 64, 64, 1, 3, [500, 77, 300], [9, 9, 130], 33, 0),
    ("bf16", 128, 64, 1, 4, [500, 77, 300], [200, 77, 130], 100, 3),
    ("fp16", 128, 16, 1, 1, [2000], [300], 10000, 0),
    # the widest window, with queries before the first token
    ("bf16", 128, 16, 1, 2, [3, 0, 20], [8, 5, 8], 2 ** 31 - 1, 0),
    ("fp16", 64, 16, 1, 1, [3, 700, 2], [9, 1, 2], 2 ** 31 - 1, 2),
    ("bf16", 128, 16, 1, 4, [3, 0, 60], [140, 33, 129], 2 ** 31 - 1, 0),
    # long ones, by the library's choice: a line of units cut anywhere, several splits
    ("bf16", 128, 64, 2, 4, [6000, 1, 900], [1, 1, 1], 0, 0),
    ("fp16", 64, 32, 1, 2, [9000, 40, 0, 2500], [8, 8, 8, 5], 0, 0),
    ("bf16", 64, 128, 1, 4, [4000, 130], [33, 20], 0, 0),
    # a wave of whole row blocks and a few that are split
    ("bf16", 64, 16, 8, 3, [2900 - 37 * b for b in range(19)], [6 - b % 2 for b in range(19)], 0, 0),
    ("fp16", 64, 32, 8, 8, [1500 - 29 * b for b in range(10)], [40 - b for b in range(10)], 0, 0),
    ("bf16", 128, 64, 8, 3, [2900 - 37 * b for b in range(19)], [6] * 19, 1500, 0),
    # more requests than lanes, and than threads of a block; empty ones among them
    ("bf16", 128, 16, 1, 2, [(b * 37) % 190 for b in range(40)], [b % 3 for b in range(40)], 0, 0),
    ("fp16", 64, 16, 2, 1, [(b * 37) % 190 for b in range(300)], [(b + 1) % 2 for b in range(300)], 0, 2),
    ("bf16", 64, 16, 1, 6, [(b * 53) % 90 for b in range(300)], [b % 6 for b in range(300)], 0, 1),
]


@pytest.mark.parametrize("dtype,D,P,Hkv,G,lens,news,window,splits", CASES)
def test_attention(dtype, D, P, Hkv, G, lens, news, window, splits):
    pages = sum(-(-a // P) for a in lens) + 3
    width = max(-(-a // P) for a in lens) + 2
    c = make(dtype, Hkv * G, Hkv, D, P, pages, width, 1, -2)
    table, kv = fill(c, dtype, lens, 11)
    if window:  # pages wholly behind every window may be gone
        tb = table.cpu().numpy()
        for b, (a, n) in enumerate(zip(lens, news)):
            tb[b, :max(0, a - n + 1 - window) // P] = -1
        table = i32(tb)
    total, scale = sum(news), D ** -0.5
    cu = i32(np.concatenate([[0], np.cumsum(news)]))
    wide = rand((total + 2, Hkv * G + 1, D), dtype, 5)
    q = wide[:total, :Hkv * G]
    out, lse = torch.full((total, Hkv * G, D), 7.0, dtype=DT[dtype], device="cuda"), torch.full((total, Hkv * G), 7.0, device="cuda")
    mq, ml = max(news), max(max(lens), 1)
    ws = torch.empty(K.kvq_paged_attention_workspace(c.cfg, len(lens), total, mq, ml, splits), dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)
    K.kvq_paged_attention(c, q, cu, i32(lens), table, mq, ml, scale, out, ws, window=window, lse=lse, splits=splits)
    assert K.kvq_paged_get_status(c) == 0
    check(out, lse, f64(q), kv, news, scale, window, dtype)
    again = torch.empty_like(out)
    K.kvq_paged_attention(c, q, cu, i32(lens), table, mq, ml, scale, again, ws, window=window, splits=splits)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))
    if all(n == 1 for n in news):  # the single-token form
        K.kvq_paged_attention(c, q, None, i32(lens), table, 1, ml, scale, again, ws, window=window, splits=splits)
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("n,splits", [(1, 0), (20, 0), (20, 1)])
def test_attention_over_millions_of_tokens(n, splits):
    """Equal weights over values of one sign, whose sums only grow.  Tolerance: the output's half
    step, and for 2^17 / 16 sums in a row at most a step of binary32 (2^-23) each."""
    T, P, D = 1 << 22, 128, 64
    c = make("fp16", 1, 1, D, P, T // P, T // P)
    v = torch.rand((T, 1, D), generator=torch.Generator("cuda").manual_seed(1), device="cuda", dtype=torch.float16) + 0.5
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    K.kvq_paged_append(c, torch.zeros_like(v), v, slots)
    kh = torch.empty_like(v)
    K.kvq_paged_dequantize(c, slots, kh, v)
    q, out, lse = rand((n, 1, D), "fp16", 2), torch.empty((n, 1, D), dtype=torch.float16, device="cuda"), torch.empty((n, 1), device="cuda")
    ws = torch.empty(max(16, K.kvq_paged_attention_workspace(c.cfg, 1, n, n, T, splits)), dtype=torch.uint8, device="cuda")
    K.kvq_paged_attention(c, q, i32([0, n]), i32([T]), slots[:T // P].view(1, -1), n, T, 1.0, out, ws, lse=lse, splits=splits)
    for i in (0, n - 1):
        seen = T - n + 1 + i
        want = v[:seen, 0].mean(0, dtype=torch.float64)
        assert ((out[i, 0].double() - want).abs() <= want * (2.0 ** -11 * 1.01 + 2.0 ** 13 * 2.0 ** -23)).all()
        assert abs(lse[i, 0].item() - np.log(seen)) <= 2.0 ** -22 * (np.log(seen) + 20)
    assert K.kvq_paged_get_status(c) == 0


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("size", [1e-30, 1e-3, 1e3])
@pytest.mark.parametrize("n", [1, 40])
def test_attention_query_sizes(dtype, size, n):
    """Tiny and large queries, one-hot softmax among them."""
    c = make(dtype, 4, 1, 128, 16, 40, 40)
    table, kv = fill(c, dtype, [333], 3)
    q = (rand((n, 4, 128), dtype, 4).float() * size).to(DT[dtype])
    out, lse = torch.empty_like(q), torch.empty((n, 4), device="cuda")
    ws = torch.empty(K.kvq_paged_attention_workspace(c.cfg, 1, n, n, 333), dtype=torch.uint8, device="cuda")
    K.kvq_paged_attention(c, q, i32([0, n]), i32([333]), table, n, 333, 0.1, out, ws, lse=lse)
    check(out, lse, f64(q), kv, [n], 0.1, 0, dtype)


@pytest.mark.parametrize("n", [1, 3, 40, 200])
def test_attention_leaves_other_rows(n):
    c = make("bf16", 4, 2, 128, 16, 40, 20)
    table, kv = fill(c, "bf16", [200, 300], 3)
    total = 2 * n + 9
    q = rand((total, 4, 128), "bf16", 4)
    out, lse = torch.full_like(q, 7.0), torch.full((total, 4), 7.0, device="cuda")
    cu = i32([2, 2 + n, 2 + 2 * n])
    ws = torch.empty(K.kvq_paged_attention_workspace(c.cfg, 2, total, n, 300, 2), dtype=torch.uint8, device="cuda")
    K.kvq_paged_attention(c, q, cu, i32([200, 300]), table, n, 300, 0.1, out, ws, lse=lse, splits=2)
    mid = slice(2, 2 + 2 * n)
    check(out[mid], lse[mid], f64(q[mid]), kv, [n, n], 0.1, 0, "bf16")
    for x in (out, lse):
        assert bool((x[:2] == 7).all()) and bool((x[2 + 2 * n:] == 7).all())


@pytest.mark.parametrize("n", [1, 5, 100])
def test_attention_bad_pages_count_as_unseen(n):
    P = 16
    c = make("bf16", 4, 1, 128, P, 30, 20)
    table, kv = fill(c, "bf16", [160], 3)
    t2 = table.clone()
    t2[0, 3], t2[0, 6], t2[0, 7] = 30, -1, 2**31 - 1
    gone = np.zeros(160, bool)
    for j in (3, 6, 7):
        gone[j * P:(j + 1) * P] = True
    q = rand((n, 4, 128), "bf16", 4)
    out = torch.empty_like(q)
    ws = torch.empty(K.kvq_paged_attention_workspace(c.cfg, 1, n, n, 160), dtype=torch.uint8, device="cuda")
    K.kvq_paged_attention(c, q, i32([0, n]), i32([160]), t2, n, 160, 0.1, out, ws)
    assert K.kvq_paged_get_status(c) == K.KVQ_STATUS_BAD_PAGE
    k, v = kv[0]
    for i in range(n):
        keep = ~gone
        keep[160 - n + i + 1:] = False
        x = np.einsum("td,hd->ht", k[keep, 0], f64(q)[i]) * 0.1
        p = np.exp(x - x.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        want, pv = p @ v[keep, 0], p @ np.abs(v[keep, 0])
        assert np.all(np.abs(f64(out)[i] - want) <= np.abs(want) * 2.0 ** -8 + pv * 2.0 ** -10)


@pytest.mark.parametrize("n", [1, 40])
def test_attention_reports_lengths_past_the_bounds(n):
    c = make("bf16", 4, 1, 128, 16, 30, 20)
    table, kv = fill(c, "bf16", [160], 3)
    q = rand((n, 4, 128), "bf16", 4)
    out = torch.empty_like(q)
    ws = torch.empty(K.kvq_paged_attention_workspace(c.cfg, 1, n, n, 100), dtype=torch.uint8, device="cuda")
    K.kvq_paged_attention(c, q, i32([0, n]), i32([160]), table, n, 100, 0.1, out, ws)
    assert K.kvq_paged_get_status(c) == K.KVQ_STATUS_LEN_OVERFLOW
    # queries stand at their true positions and see only the first 100 tokens
    k, v = kv[0][0][:100], kv[0][1][:100]
    o, _, pv, _ = R.attention(f64(q).reshape(1, n * 4, 128), k, v, 1, 0.1, 0)
    want, pv = o.reshape(n, 4, 128), pv.reshape(n, 4, 128)
    assert np.all(np.abs(f64(out) - want) <= np.abs(want) * 2.0 ** -8 + pv * 2.0 ** -10)


@pytest.mark.parametrize("scale", [-0.07, 0.0, 30.0])
@pytest.mark.parametrize("n", [1, 40])
def test_attention_scales(scale, n):
    for dtype in ("fp16", "bf16"):
        c = make(dtype, 4, 1, 128, 16, 40, 40)
        table, kv = fill(c, dtype, [333], 3)
        q = rand((n, 4, 128), dtype, 4)
        out, lse = torch.empty_like(q), torch.empty((n, 4), device="cuda")
        ws = torch.empty(max(16, K.kvq_paged_attention_workspace(c.cfg, 1, n, n, 333)), dtype=torch.uint8, device="cuda")
        K.kvq_paged_attention(c, q, i32([0, n]), i32([333]), table, n, 333, scale, out, ws, lse=lse)
        check(out, lse, f64(q), kv, [n], scale, 0, dtype)


@pytest.mark.parametrize("splits", [0, 2])
def test_attention_nan_query_stays_in_its_row(splits):
    for n in (1, 6, 100):
        c = make("bf16", 4, 1, 128, 16, 30, 20)
        table, kv = fill(c, "bf16", [160], 3)
        q = rand((n, 4, 128), "bf16", 4)
        q[0, 2, 5] = float("nan")
        out = torch.empty_like(q)
        ws = torch.empty(max(16, K.kvq_paged_attention_workspace(c.cfg, 1, n, n, 160, splits)), dtype=torch.uint8, device="cuda")
        K.kvq_paged_attention(c, q, i32([0, n]), i32([160]), table, n, 160, 0.1, out, ws, splits=splits)
        bad = torch.isnan(out).any(-1)
        assert bool(bad[0, 2]) and int(bad.sum()) == 1


# ------------------------------------------------------------------------------ together
def serve(cfg, steps, layers=2, finish=None):
    """Rounds of a session over requests of changing lengths, every layer against 64 bits."""
    B, D = len(steps[0]), cfg.D
    rope = K.make_rope_cfg(cfg.Hq, cfg.Hkv, D, D, [0] * (D // 2), torch.bfloat16)
    freqs = 1e4 ** (-torch.arange(D // 2, dtype=torch.float64, device="cuda") / (D // 2))
    s = PagedSession(cfg, layers, B, rope, freqs)
    for c in s.caches:
        c.pool.fill_(0xFF)
    hist = [[([np.zeros((0, cfg.Hkv, D))], [np.zeros((0, cfg.Hkv, D))]) for _ in range(B)] for _ in range(layers)]
    for step, new in enumerate(steps):
        n = sum(new)
        s.begin(i32(new), n, max(new))
        for layer in range(layers):
            qkv = rand((n, cfg.Hq + 2 * cfg.Hkv, D), "bf16", 100 * layer + step)
            q, k, v = qkv[:, :cfg.Hq], qkv[:, cfg.Hq:cfg.Hq + cfg.Hkv], qkv[:, cfg.Hq + cfg.Hkv:]
            raw = k.clone()
            out = torch.empty((n, cfg.Hq, D), dtype=torch.bfloat16, device="cuda")
            s.attend(layer, q, k, v, D ** -0.5, out)
            # the rotated keys, within the rotation's tolerance, are what is stored
            at, h = 0, hist[layer]
            pos = s.positions.cpu().numpy()
            angle = pos[:, None].astype(np.float64) * freqs.cpu().numpy()
            cs, sn = np.cos(angle)[:, None], np.sin(angle)[:, None]
            u, w = f64(raw)[..., :D // 2], f64(raw)[..., D // 2:]
            turned = np.concatenate([u * cs - w * sn, w * cs + u * sn], -1)
            assert np.all(np.abs(f64(k) - turned) <= np.abs(turned) * 2.0 ** -8 + 2.0 ** -18 * (np.abs(u) + np.abs(w)).repeat(2, -1).max())
            for b, m in enumerate(new):
                h[b][0].append(R.quantize(f64(k[at:at + m])))
                h[b][1].append(R.quantize(f64(v[at:at + m])))
                at += m
            kv = [(np.concatenate(a), np.concatenate(z)) for a, z in h]
            assert s.lens.tolist() == [len(a) for a, _ in kv]
            check(out, None, f64(q), kv, new, D ** -0.5, 0, "bf16")
        if finish and step in finish:
            s.finish(i32([b in finish[step] for b in range(B)]))
            for layer in range(layers):
                for b in finish[step]:
                    hist[layer][b] = ([np.zeros((0, cfg.Hkv, D))], [np.zeros((0, cfg.Hkv, D))])
    assert s.status() == 0


@pytest.mark.parametrize("P", [16, 64])
def test_serving_rounds(P):
    cfg = K.make_paged_cfg(8, 2, 128, P, 60 * 16 // P, 20 * 16 // P, torch.bfloat16)
    serve(cfg, [[40, 1, 0, 17, 150], [1, 1, 1, 1, 1], [1, 30, 64, 1, 1], [4, 4, 4, 4, 4], [1] * 5, [100, 1, 1, 0, 1], [1] * 5], finish={3: [0, 4], 4: [2]})


def test_serving_on_another_stream():
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        serve(K.make_paged_cfg(4, 1, 128, 32, 60, 12, torch.bfloat16), [[30, 5, 9, 1, 2], [1, 1, 1, 1, 1]])
    s.synchronize()


@pytest.mark.parametrize("n,lens0,splits", [(1, [14, 40, 0], 0), (1, [14, 40, 0], 3), (3, [2000, 40, 16], 0), (20, [14, 300, 0], 0), (20, [14, 300, 0], 2)])
def test_captured_step_replays(n, lens0, splits):
    """A step as a CUDA graph: plan, append and attention in place, replayed as lengths grow."""
    B, P, Hq, Hkv, D, rounds = 3, 16, 4, 2, 128, 6
    pages, width = 200, 140
    c = make("bf16", Hq, Hkv, D, P, pages, width)
    table, kv = fill(c, "bf16", lens0, 3)
    used = sum(-(-a // P) for a in lens0)
    free = i32(np.concatenate([np.random.RandomState(3).permutation(pages)[used:], np.zeros(used)]))
    n_free, lens, new = i32([pages - used]), i32(lens0), i32([n] * B)
    q, k, v = (torch.empty((n * B, h, D), dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
    out, lse = torch.empty_like(q), torch.empty((n * B, Hq), device="cuda")
    cu, slots, pos = i32([0] * (B + 1)), i32([0] * n * B), i32([0] * n * B)
    ws = torch.empty(max(16, K.kvq_paged_attention_workspace(c.cfg, B, n * B, n, width * P, splits)), dtype=torch.uint8, device="cuda")

    def step():
        K.kvq_page_plan(c, lens, new, table, free, n_free, cu, lens, n_free, slots, pos)
        K.kvq_paged_append(c, k, v, slots)
        K.kvq_paged_attention(c, q, cu, lens, table, n, width * P, 0.1, out, ws, lse=lse, splits=splits)

    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    hist = [[a, z] for a, z in kv]
    for r in range(rounds):
        for x, seed in ((q, 1), (k, 2), (v, 3)):
            x.copy_(rand(x.shape, "bf16", 50 * r + seed))
        if r == 2:
            step()  # the same, launched one by one
        else:
            g.replay()
        for b in range(B):
            at = slice(n * b, n * b + n)
            hist[b] = [np.concatenate([hist[b][i], R.quantize(f64(x[at]))]) for i, x in enumerate((k, v))]
        assert lens.tolist() == [a + n * (r + 1) for a in lens0]
        check(out, lse, f64(q), hist, [n] * B, 0.1, 0, "bf16")
    assert K.kvq_paged_get_status(c) == 0


def test_two_streams_at_once():
    """Decode, drafts and chunks of two batches on two streams, each with its own workspace."""
    runs = []
    for n, splits, seed in ((1, 3, 1), (4, 0, 2), (70, 2, 3)):
        c = make("bf16", 8, 2, 128, 32, 300, 100)
        lens = [3000, 77, 1500]
        table, kv = fill(c, "bf16", lens, seed)
        q = rand((3 * n, 8, 128), "bf16", seed + 9)
        cu, ln = i32([0, n, 2 * n, 3 * n]), i32(lens)
        ws = torch.empty(K.kvq_paged_attention_workspace(c.cfg, 3, 3 * n, n, 3000, splits), dtype=torch.uint8, device="cuda")
        alone = torch.empty_like(q)
        call = lambda out, c=c, q=q, cu=cu, ln=ln, table=table, n=n, ws=ws, splits=splits: K.kvq_paged_attention(  # noqa: E731
            c, q, cu, ln, table, n, 3000, 0.1, out, ws, splits=splits)
        call(alone)
        runs.append((call, alone, torch.empty_like(q), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for call, _, out, s in runs:
            with torch.cuda.stream(s):
                call(out)
    torch.cuda.synchronize()
    for _, alone, out, _ in runs:
        assert torch.equal(alone.view(torch.int16), out.view(torch.int16))
