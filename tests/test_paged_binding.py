"""What the paged cache's binding does before and around the library's calls (no GPU)."""
import contextlib

import pytest
import torch

import long_context_decode_nuq_b200 as K
from long_context_decode_nuq_b200 import kvq


def test_status_is_read_on_the_caches_device(monkeypatch):
    """A cache of device 3 while device 0 is current: the call runs on device 3 and its stream (the
    default stream's handle is 0 on every device, and means the current one's)."""
    c = K.PagedCache(K.make_paged_cfg(8, 2, 128, 16, 10, 4, torch.bfloat16), device="cpu")
    c.index, c.device = 3, torch.device("cuda", 3)
    current, seen = [0], []

    @contextlib.contextmanager
    def on(i):
        old, current[0] = current[0], i
        yield
        current[0] = old

    class Lib:
        def kvq_paged_get_status(self, cache, out, stream):
            seen.append((current[0], stream))
            out._obj.value = 128
            return 0

    kvq._torch()
    monkeypatch.setattr(kvq, "load", Lib)
    monkeypatch.setattr(kvq, "_current", lambda: current[0])
    monkeypatch.setattr(kvq, "_raw_stream", lambda i: 1000 + i)
    monkeypatch.setattr(torch.cuda, "device", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: type("S", (), {"cuda_stream": 1000 + d.index}))
    assert K.kvq_paged_get_status(c) == 128
    assert seen == [(3, 1003)] and current[0] == 0


def test_rope_cfg_filled_by_hand():
    """kvq_rope takes a RopeCfg that make_rope_cfg did not make: it says what is wrong with the
    tensors (here: host memory), from the struct's own fields."""
    axes = [0, 1] * 8
    a = K.make_rope_cfg(2, 1, 64, 32, axes, torch.bfloat16)
    b = K.RopeCfg(2, 1, 64, 32, 1, 0, 2, a.pair_axis)
    q, k, pos, freqs = torch.zeros((3, 2, 64)).bfloat16(), torch.zeros((3, 1, 64)).bfloat16(), torch.zeros((2, 3), dtype=torch.int32), torch.zeros(16).double()
    for cfg in (a, b):
        with pytest.raises(ValueError, match="not on a CUDA device"):
            K.kvq_rope(cfg, q, k, pos, freqs, q, k)
        with pytest.raises(ValueError, match="positions"):
            K.kvq_rope(cfg, q, k, pos[:1], freqs, q, k)
        with pytest.raises(ValueError, match="q is"):
            K.kvq_rope(cfg, q.half(), k, pos, freqs, q, k)
    with pytest.raises(ValueError, match="float16, bfloat16 or float32"):
        K.kvq_rope(K.RopeCfg(2, 1, 64, 32, 7, 0, 2, a.pair_axis), q, k, pos, freqs, q, k)


def test_session_begins_a_step_without_tokens():
    """A step in which no request brings a token: refused only for its host memory, which comes last."""
    from long_context_decode_nuq_b200.paged import PagedSession
    s = PagedSession(K.make_paged_cfg(4, 2, 64, 16, 40, 20, torch.bfloat16), 1, 2, device="cpu")
    with pytest.raises(ValueError, match="not on a CUDA device"):
        s.begin(torch.zeros(2, dtype=torch.int32), 0, 0)
    assert s.slots.numel() == s.positions.numel() == 0


def test_plan_list_refuses_a_negative_size():
    import ctypes
    c = K.PagedCache(K.make_paged_cfg(1, 1, 64, 16, 10, 4, torch.bfloat16), device="cpu")
    a = (ctypes.addressof((ctypes.c_uint8 * 512)()) + 255) & ~255
    plan = K.load().kvq_page_plan_list
    assert plan(*c.args, 3, a, a, a, a, -1, a, 7, a, a, a, a, a, None) == -3
    assert plan(*c.args, 3, a, a, a, None, 5, a, 7, a, a, a, a, a, None) == -1


@pytest.mark.parametrize("change", [dict(window=(1 << 32) + 5), dict(max_len=(1 << 32) + 64), dict(max_q=1 << 32 | 1), dict(splits=1 << 33),
                                    dict(window=-(1 << 32))])
def test_sizes_past_32_bits_are_refused(change):
    """They would be cut to 32 bits on the way to the library: a window of 2^32 + 5 became 5."""
    c = K.PagedCache(K.make_paged_cfg(8, 2, 128, 16, 10, 4, torch.bfloat16), device="cpu")
    i = lambda *s: torch.zeros(s, dtype=torch.int32)  # noqa: E731
    q = torch.zeros((3, 8, 128)).bfloat16()
    kw = {**dict(max_q=1, max_len=64, window=0, splits=0), **change}
    with pytest.raises(ValueError, match="32 bits"):
        K.kvq_paged_attention(c, q, None, i(3), i(3, 4), sm_scale=0.1, out=q, **kw)
    if "window" not in change:
        kw.pop("window")
        with pytest.raises(ValueError, match="32 bits"):
            K.kvq_paged_attention_workspace(c.cfg, 3, 3, **kw)


@pytest.mark.parametrize("change", [dict(num_pages=(1 << 32) + 10), dict(max_pages=1 << 32 | 4), dict(Hq=(1 << 32) + 8), dict(k_exp=1 << 32)])
def test_configurations_past_32_bits_are_refused(change):
    with pytest.raises(ValueError, match="32 bits"):
        K.make_paged_cfg(**{**dict(Hq=8, Hkv=2, D=128, page_tokens=16, num_pages=10, max_pages=4, dtype=torch.bfloat16), **change})
    if "Hq" in change:
        with pytest.raises(ValueError, match="32 bits"):
            K.make_rope_cfg(change["Hq"], 2, 128, 128, [0] * 64, torch.bfloat16)
