"""Arguments that the paged cache's calls and kvq_rope refuse before anything is launched."""
import ctypes

import pytest
import torch

import long_context_decode_nuq_b200 as K

OK = dict(Hq=8, Hkv=2, D=128, page_tokens=16, num_pages=10, max_pages=4, dtype=1, k_exp=0, v_exp=0)
NULL, ALIGN, SHAPE, UNSUPPORTED, RANGE, WORKSPACE = -1, -2, -3, -4, -5, -6
MEM = (ctypes.c_uint8 * 4096)()
A = (ctypes.addressof(MEM) + 255) & ~255  # an aligned address; nothing is read from it


def cfg(**kw):
    return K.PagedCfg(*{**OK, **kw}.values())


@pytest.mark.parametrize("kw,code", [
    ({}, 0), (dict(D=96), UNSUPPORTED), (dict(page_tokens=48), UNSUPPORTED), (dict(page_tokens=256), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
    (dict(Hkv=0), SHAPE), (dict(Hkv=3), SHAPE), (dict(Hq=1), SHAPE), (dict(Hq=130), SHAPE), (dict(num_pages=0), SHAPE), (dict(max_pages=0), SHAPE),
    (dict(num_pages=1 << 27), SHAPE), (dict(max_pages=1 << 27), SHAPE), (dict(max_pages=(1 << 27) - 256), SHAPE), (dict(max_pages=(1 << 27) - 257), 0),
    (dict(k_exp=65), RANGE), (dict(v_exp=-65), RANGE)])
def test_config(kw, code):
    c = cfg(**kw)
    assert K.kvq_paged_validate_cfg(c) == code
    n = ctypes.c_size_t()
    assert K.load().kvq_paged_layout(ctypes.byref(c), ctypes.byref(n)) == code
    if code == 0:
        assert n.value == 10 * 2 * 16 * 2 * (64 + 8)


def cache(pool=A, status=A):
    return ctypes.byref(K.PagedStruct(pool, status))


def call(name, *args):
    return getattr(K.load(), name)(*args)


@pytest.mark.parametrize("change,code", [
    ({1: None}, NULL), ({1: cache(None)}, NULL), ({1: cache(A + 8)}, ALIGN), ({2: None}, NULL), ({2: A + 2}, ALIGN), ({4: None}, NULL),
    ({3: 252}, ALIGN), ({3: 248}, SHAPE), ({5: 260}, ALIGN), ({5: 128}, SHAPE), ({6: None}, NULL), ({7: -1}, SHAPE), ({7: 0}, 0)])
def test_append(change, code):
    a = [ctypes.byref(cfg()), cache(), A, 256, A, 256, A, 5, None]
    for i, x in change.items():
        a[i] = x
    assert call("kvq_paged_append", *a) == code


@pytest.mark.parametrize("change,code", [({2: None}, NULL), ({3: -2}, SHAPE), ({4: A + 4}, ALIGN), ({5: None}, NULL), ({3: 0}, 0)])
def test_dequantize(change, code):
    a = [ctypes.byref(cfg()), cache(), A, 5, A, A, None]
    for i, x in change.items():
        a[i] = x
    assert call("kvq_paged_dequantize", *a) == code


@pytest.mark.parametrize("change,code", [
    ({1: None}, NULL), ({2: 0}, SHAPE), ({2: (1 << 20) + 1}, SHAPE), ({3: None}, NULL), ({5: None}, NULL), ({8: -1}, SHAPE), ({8: (1 << 30) + 1}, SHAPE), ({9: None}, NULL),
    ({12: None}, NULL), ({13: None}, NULL)])
def test_plan(change, code):
    a = [ctypes.byref(cfg()), cache(), 3, A, A, A, A, A, 7, A, A, A, A, A, None]
    for i, x in change.items():
        a[i] = x
    assert call("kvq_page_plan", *a) == code


@pytest.mark.parametrize("change,code", [({1: None}, NULL), ({2: 0}, SHAPE), ({3: None}, NULL), ({4: None}, NULL), ({7: None}, NULL)])
def test_release(change, code):
    a = [ctypes.byref(cfg()), cache(), 3, A, A, A, A, A, None]
    for i, x in change.items():
        a[i] = x
    assert call("kvq_page_release", *a) == code


@pytest.mark.parametrize("change,code", [
    ({1: None}, NULL), ({2: None}, NULL), ({2: A + 8}, ALIGN), ({3: 1020}, ALIGN), ({3: 1016}, SHAPE), ({4: None}, SHAPE), ({5: 0}, SHAPE),
    ({5: 70000}, SHAPE), ({6: -1}, SHAPE), ({6: 0}, 0), ({7: None}, NULL), ({8: None}, NULL), ({9: 0}, SHAPE), ({10: 0}, SHAPE),
    ({11: float("nan")}, RANGE), ({11: float("inf")}, RANGE), ({11: 3e38}, RANGE), ({12: -1}, RANGE), ({13: A + 2}, ALIGN), ({13: None}, NULL), ({15: None}, NULL),
    ({15: A + 8}, ALIGN), ({16: 10}, WORKSPACE), ({17: 257}, RANGE), ({17: -1}, RANGE)])
def test_attention(change, code):
    a = [ctypes.byref(cfg()), cache(), A, 1024, A, 3, 9, A, A, 4, 640, 0.1, 0, A, None, A, 1 << 30, 2, None]
    for i, x in change.items():
        a[i] = x
    assert call("kvq_paged_attention", *a) == code


def test_workspace_sizes():
    # 16 rows a kv head: pieces of two per block, and a count per request
    n = [K.kvq_paged_attention_workspace(cfg(), 3, 9, 4, 5000, s) for s in (0, 1, 2, 256)]
    assert n[1] == 2 * 6 * 16 * 130 * 4 + 6 * 16 and n[1] < n[2] < n[0] < n[3]
    # 800 rows: splits of all rows
    n = [K.kvq_paged_attention_workspace(cfg(), 3, 600, 200, 5000, s) for s in (1, 2, 256)]
    assert n == [0, 2 * 600 * 8 * 130 * 4, 256 * 600 * 8 * 130 * 4]
    assert K.kvq_paged_attention_workspace(cfg(), 3, 3, 1, 64) == 0
    # and no split of more than 2^17 tokens
    wide = cfg(max_pages=1 << 16)
    n = [K.kvq_paged_attention_workspace(wide, 3, 600, 200, t, 1) for t in (1 << 17, (1 << 17) + 1, 1 << 20)]
    assert n == [0, 2 * 600 * 8 * 130 * 4, 8 * 600 * 8 * 130 * 4]


@pytest.mark.parametrize("kw,change,code", [
    ({}, {1: None}, NULL), ({}, {1: A + 2}, ALIGN), ({}, {2: 1028}, ALIGN), ({}, {2: 1016}, SHAPE), ({}, {3: None}, NULL), ({}, {4: 248}, SHAPE),
    ({}, {5: None}, NULL), ({}, {6: None}, NULL), ({}, {6: A + 4}, ALIGN), ({}, {7: -1}, SHAPE), ({}, {7: 0}, 0), ({}, {8: 2}, SHAPE),
    ({}, {9: None}, NULL), ({}, {9: A, 10: 2048}, SHAPE), ({}, {11: None}, NULL), (dict(D=24), {}, UNSUPPORTED), (dict(rot_dim=144), {}, UNSUPPORTED),
    (dict(rot_dim=8), {}, UNSUPPORTED), (dict(dtype=3), {}, UNSUPPORTED), (dict(Hq=0), {}, SHAPE), (dict(axes=0), {}, SHAPE), (dict(axes=9), {}, SHAPE),
    (dict(adjacent=2), {}, SHAPE), (dict(axes=2), {}, RANGE)])
def test_rope(kw, change, code):
    c = K.RopeCfg(8, 2, 128, 128, 1, 0, 3, (ctypes.c_uint8 * 128)(*([2] * 64)))
    for f, x in kw.items():
        setattr(c, f, x)
    a = [ctypes.byref(c), A, 1024, A, 256, A, A, 5, 0, A + 512, 1024, A + 512, 256, None]
    for i, x in change.items():
        a[i] = x
    assert call("kvq_rope", *a) == code


def test_binding_checks_tensors():
    """What the binding sees before the library does (tensors in host memory)."""
    c = K.PagedCache(cfg(), pool=torch.empty(K.kvq_paged_layout(cfg()), dtype=torch.uint8))
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    h = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    bad = [
        lambda: K.PagedCache(cfg(), pool=torch.empty(7, dtype=torch.uint8)),
        lambda: K.make_paged_cfg(8, 2, 128, 16, 10, 4, torch.float64),
        lambda: K.kvq_paged_append(c, h(5, 2, 128), h(5, 2, 64), i(5)),
        lambda: K.kvq_paged_append(c, h(5, 2, 128).half(), h(5, 2, 128), i(5)),
        lambda: K.kvq_paged_append(c, h(5, 2, 128), h(5, 2, 128), i(5).long()),
        lambda: K.kvq_paged_append(c, h(5, 128, 2).transpose(1, 2), h(5, 2, 128), i(5)),
        lambda: K.kvq_paged_append(c, h(5, 2, 128), h(5, 2, 128), i(5)),  # host memory
        lambda: K.kvq_paged_dequantize(c, i(5), h(5, 3, 128)[:, :2], h(5, 2, 128)),
        lambda: K.kvq_paged_attention(c, h(3, 8, 128), None, i(3), i(3, 5), 1, 64, 0.1, h(3, 8, 128)),
        lambda: K.kvq_paged_attention(c, h(3, 8, 128), i(3), i(3), i(3, 4), 1, 64, 0.1, h(3, 8, 128)),
        lambda: K.kvq_paged_attention(c, h(3, 8, 128), None, i(3), i(3, 4), 1, 64, 0.1, h(3, 8, 128), lse=h(3, 8)),
        lambda: K.kvq_page_plan(c, i(3), i(2), i(3, 4), i(10), i(1), i(4), i(3), i(1), i(9), i(9)),
        lambda: K.kvq_page_plan(c, i(3), i(3), i(3, 4), i(10), i(1), i(4), i(3), i(1), i(9), i(8)),
        lambda: K.kvq_page_release(c, i(3), i(3), i(3, 4), i(9), i(1)),
        lambda: K.make_rope_cfg(8, 2, 128, 128, [0] * 63, torch.float16),
        lambda: K.make_rope_cfg(8, 2, 128, 128, [9] * 64, torch.float16),
        lambda: K.kvq_rope(K.make_rope_cfg(8, 2, 128, 128, [0] * 64, torch.float16), h(3, 8, 128).half(), h(3, 2, 128).half(), i(1, 3),
                           torch.zeros(64), h(3, 8, 128).half(), h(3, 2, 128).half()),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()
    for kw in (dict(D=96), dict(page_tokens=17)):
        with pytest.raises(K.KvqError):
            K.make_paged_cfg(**{**{k: v for k, v in OK.items() if k != "dtype"}, **kw}, dtype=torch.float16)
