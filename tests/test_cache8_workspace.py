"""Attention over the 8-bit cache needs no workspace: its size is 0 for every problem, and a call without one is a call like any
other."""
import pytest
import torch

import chunk_wise_hierarchical_hils_b200 as hils


@pytest.mark.parametrize("kw", [dict(N=256, T=256, k=4), dict(N=1, T=4096, q_offset=4095, k=32), dict(N=4096, T=4096, k=16),
                                dict(N=1, T=1, k=0), dict(N=3, T=70, q_offset=60, k=64, d=64, C=32, in_dtype=hils.HILS_F32)])
def test_the_size_is_zero(kw):
    p = hils.problem(**dict(dict(B=2, H=8, Hkv=2, d=128, C=64), **kw))
    assert hils.hils_chunk_attend_fuse_q8_workspace_size(p) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(2, 8, 2, 1, 1000, 128, 64, 7, 900), (1, 4, 1, 7, 300, 64, 32, 3, 290),
                                   (1, 8, 2, 512, 512, 128, 64, 4, 0)], ids=lambda s: "x".join(map(str, s)))
def test_a_call_without_one(shape):
    import test_cache8_gpu as c8
    p, h, dev = c8.attend_case(*shape, "bf16", "bf16", 670)
    want, O = c8.attend(p, dev), torch.full_like(dev["Q"], 7.0)
    for ws in (None, (None, 0)):
        O.fill_(7.0)
        hils.hils_chunk_attend_fuse_q8(p, dev["Q"], dev["K8"], dev["V8"], dev["ks"], dev["vs"], dev["sel"], dev["score"], O, ws)
        c8.ok()
        assert torch.equal(O.view(torch.int16), want.view(torch.int16))
    c8.compare(p, h, O, "bf16", rows=range(0, p.N, max(1, p.N // 11)))
