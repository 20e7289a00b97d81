"""PagedSession: a captured step stays valid while steps of other sizes come between its replays."""
import pytest
import torch

import long_context_decode_nuq_b200 as K
from long_context_decode_nuq_b200.paged import PagedSession


def test_buffers_that_a_captured_step_uses_are_kept():
    """On host memory: the plan itself refuses, after begin() has found its buffers."""
    s = PagedSession(K.make_paged_cfg(4, 2, 64, 16, 400, 200, torch.bfloat16), 1, 2, device="cpu")
    n_new = torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="no step has begun"):
        s.attend(0, None, None, None, 1.0, None)
    seen = []
    for tokens, max_q in ((2, 1), (2, 2), (40, 30), (900, 600), (40, 30), (2, 1)):
        with pytest.raises(ValueError, match="not on a CUDA device"):
            s.begin(n_new, tokens, max_q)
        assert s.slots.numel() == s.positions.numel() == tokens
        assert s.workspace.numel() >= K.kvq_paged_attention_workspace(s.cfg, 2, tokens, max_q, 200 * 16)
        seen += [s.slots.data_ptr(), s.positions.data_ptr(), s.workspace.data_ptr()]
    held = {t.data_ptr() for t in [*s._held.values(), *s._outgrown]}
    assert held == set(seen)
    assert sum(t.nbytes for t in s._outgrown) <= sum(t.nbytes for t in s._held.values())


@pytest.mark.gpu
def test_captured_step_between_other_steps():
    """Two captured decode steps with different bounds, with prompts and drafts between replays:
    the same bits as a session that runs the same steps one by one."""
    cfg = K.make_paged_cfg(8, 2, 128, 16, 1500, 500, torch.bfloat16)
    B, D = 3, 128
    rope = K.make_rope_cfg(8, 2, D, D, [0] * (D // 2), torch.bfloat16)
    freqs = 1e4 ** (-torch.arange(D // 2, dtype=torch.float64, device="cuda") / (D // 2))
    a, b = (PagedSession(cfg, 2, B, rope, freqs) for _ in range(2))
    i32 = dict(dtype=torch.int32, device="cuda")
    one = torch.ones(B, **i32)

    def inputs(n, seed):
        g = torch.Generator("cuda").manual_seed(seed)
        return [torch.randn((n, h, D), generator=g, device="cuda").bfloat16() for h in (8, 2, 2) * 2]

    def step(s, new, n, max_q, max_len, x, outs):
        s.begin(new, n, max_q, max_len)
        for layer in range(2):
            s.attend(layer, *x[3 * layer:3 * layer + 3], D ** -0.5, outs[layer])

    def empty(n):
        return [torch.zeros((n, 8, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    graphs = []
    for max_len in (64, 0):
        g, x, outs = torch.cuda.CUDAGraph(), inputs(B, 1), empty(B)
        with torch.cuda.graph(g):
            step(a, one, B, 1, max_len, x, outs)
        graphs.append((g, x, outs))
    for seed, new in enumerate(([20, 1, 7], 0, [4, 4, 4], 1, [300, 1, 900], 1, [4, 4, 0], 1, [2000, 30, 1], 1, 1)):
        if isinstance(new, int):  # replay
            g, x, outs = graphs[new]
            for t, src in zip(x, inputs(B, seed)):
                t.copy_(src)
            g.replay()
            n, q, ml, new = B, 1, 64 if new == 0 else 0, [1] * B
        else:
            n, q, ml = sum(new), max(new), 0
            outs = empty(n)
            step(a, torch.tensor(new, **i32), n, q, 0, inputs(n, seed), outs)
        want = empty(n)
        step(b, torch.tensor(new, **i32), n, q, ml, inputs(n, seed), want)
        for got, w in zip(outs, want):
            assert torch.equal(got.view(torch.int16), w.view(torch.int16))
    assert a.lens.tolist() == b.lens.tolist()
    assert a.status() == b.status() == 0
