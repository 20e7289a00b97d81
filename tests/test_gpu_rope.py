"""kvq_rope against the formula in 64 bits."""
import numpy as np
import pytest
import torch

import long_context_decode_nuq_b200 as K

pytestmark = pytest.mark.gpu
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


def reference(x, pos, freqs, axis, rot, adjacent, inverse):
    x = x.double().cpu().numpy().copy()
    a = pos.cpu().numpy().astype(np.float64)[axis].T * freqs.cpu().numpy()  # [n, rot/2]
    c, s = np.cos(a)[:, None], np.sin(a)[:, None] * (-1 if inverse else 1)
    h = rot // 2
    i, j = (slice(0, rot, 2), slice(1, rot, 2)) if adjacent else (slice(0, h), slice(h, rot))
    u, v = x[..., i].copy(), x[..., j].copy()
    x[..., i], x[..., j] = u * c - v * s, v * c + u * s
    size = np.zeros_like(x)
    size[..., i] = size[..., j] = np.abs(u) + np.abs(v)
    return x, size


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("n,Hq,Hkv,D,rot,axes,top", [
    (1, 1, 0, 16, 16, 1, 10), (1, 32, 8, 128, 128, 3, 2**31 - 1), (7, 5, 3, 128, 64, 2, 1 << 20), (295, 3, 1, 64, 64, 3, 5000),
    (297, 8, 2, 256, 192, 4, 1 << 24), (2371, 4, 2, 128, 128, 3, 1 << 20), (2400, 2, 2, 80, 48, 1, 3000)])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(dtype, n, Hq, Hkv, D, rot, axes, top, adjacent, inverse):
    g = torch.Generator("cuda").manual_seed(n)
    wide = torch.randn((n, Hq + Hkv + 2, D), generator=g, device="cuda").to(DT[dtype])
    q, k = wide[:, :Hq], wide[:, Hq + 1:Hq + 1 + Hkv]
    axis = [i * 7 % axes for i in range(rot // 2)]
    axis[-1] = axes - 1
    pos = torch.randint(0, top, (axes, n), generator=g, device="cuda").int()
    freqs = 1e4 ** (-torch.arange(rot // 2, dtype=torch.float64, device="cuda") / (rot // 2))
    cfg = K.make_rope_cfg(Hq, Hkv, D, rot, axis, DT[dtype], adjacent=adjacent)
    qo = torch.empty((n, Hq, D), dtype=DT[dtype], device="cuda")
    ko = torch.empty((n, Hkv, D), dtype=DT[dtype], device="cuda") if Hkv else None
    K.kvq_rope(cfg, q, k if Hkv else None, pos, freqs, qo, ko, inverse=inverse)
    # the output's rounding; binary32: the angle's remainder (2^-23 of pi at most), cos and sin (two
    # units each), two products and a sum, all relative to |u| + |v|
    for x, y in ((q, qo), (k, ko))[:2 if Hkv else 1]:
        want, size = reference(x, pos, freqs, axis, rot, adjacent, inverse)
        got = y.double().cpu().numpy()
        tol = np.abs(want) * float(torch.finfo(DT[dtype]).eps) / 2 * 1.01 + size * 6 * 2.0 ** -23 + (2.0 ** -25 if dtype == "fp16" else 0)
        assert np.all(np.abs(got - want) <= tol)
        assert np.array_equal(got[..., rot:], x.double().cpu().numpy()[..., rot:])
    # in place, rows of the wider projection
    if Hkv:
        edge = wide[:, [Hq, Hq + 1 + Hkv]].clone()
        K.kvq_rope(cfg, q, k, pos, freqs, q, k, inverse=inverse)
        assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(edge, wide[:, [Hq, Hq + 1 + Hkv]])


def test_inverse_is_the_gradient():
    """d<w, rope(x)>/dx by differences equals rope(w, inverse)."""
    n, H, D = 5, 2, 64
    g = torch.Generator("cuda").manual_seed(1)
    x, w, e = (torch.randn((n, H, D), generator=g, device="cuda") for _ in range(3))
    pos = torch.randint(0, 9000, (3, n), generator=g, device="cuda").int()
    freqs = 1e4 ** (-torch.arange(32, dtype=torch.float64, device="cuda") / 32)
    cfg = K.make_rope_cfg(H, 0, D, D, [i % 3 for i in range(32)], torch.float32)
    out = lambda y, inv: (z := torch.empty_like(y), K.kvq_rope(cfg, y, None, pos, freqs, z, None, inverse=inv))[0]  # noqa: E731
    step = ((out(x + e, False).double() - out(x - e, False).double()) * w).sum() / 2  # the map is linear
    grad = out(w, True).double()
    # n H D = 640 terms of about 1, each right to 2^-21
    assert abs(float(step - (grad * e).sum())) <= 640 * 8 * 2.0 ** -21
