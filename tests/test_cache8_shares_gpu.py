"""Every instance of the 8-bit cache's row attention under every way of sharing a row out: the head dimension, the chunk, the
types and whether a warp, a block or a cluster of blocks takes a row of work are each compiled or laid out for themselves, and
the rule that chooses among the latter would reach only some of them at a test's sizes."""
import numpy as np
import pytest
import torch

import test_cache8_gpu as c8

pytestmark = pytest.mark.gpu

TYPES = [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")]
SHARES = [0, 1, 2, 5, 8]


def shape(d, C, G, N=5, k=11, B=2, Hkv=2):
    """A few queries on both sides of a chunk's start, more past chunks than slots, room behind the last token."""
    q0 = 14 * C - 3
    return B, G * Hkv, Hkv, N, q0 + N + 70, d, C, k, q0


@pytest.mark.parametrize("share", SHARES)
@pytest.mark.parametrize("dtype,out", TYPES)
@pytest.mark.parametrize("d,C", [(64, 32), (64, 64), (64, 128), (128, 32), (128, 64), (128, 128)])
def test_every_instance_and_share(d, C, dtype, out, share, monkeypatch):
    monkeypatch.setenv("HILS_Q8_KERNEL", "rows")
    monkeypatch.setenv("HILS_Q8_SHARE", str(share))
    for G in (3, 12):                                       # a group within a row of work, and one of two or three rows
        p, h, dev = c8.attend_case(*shape(d, C, G), dtype, out, 800 + d + C + G)
        O = c8.attend(p, dev)
        O2 = c8.attend(p, dev)
        c8.ok()
        assert torch.equal(O.view(torch.uint8), O2.view(torch.uint8))
        c8.compare(p, h, O, out)


@pytest.mark.parametrize("share", range(9))
@pytest.mark.parametrize("k,q0", [(0, 3), (1, 70), (2, 64), (64, 64 * 80 + 5)])
def test_fewer_or_more_turns_than_warps(k, q0, share, monkeypatch):
    """Rows of one slot, of less than a warp each, and of the most there can be; some slots empty."""
    monkeypatch.setenv("HILS_Q8_KERNEL", "rows")
    monkeypatch.setenv("HILS_Q8_SHARE", str(share))

    def edit(h, r):
        h["sel"][:, :, ::2, ::3] = -1
    p, h, dev = c8.attend_case(1, 8, 2, 3, q0 + 3, 128, 64, k, q0, "bf16", "bf16", 820 + k, edit=edit)
    O = c8.attend(p, dev)
    c8.ok()
    c8.compare(p, h, O, "bf16")


@pytest.mark.parametrize("shape,dtype,share", [
    ((1, 2, 2, 1003, 1024, 64, 32, 4, 0), "f32", 0), ((16, 32, 8, 4, 700, 128, 64, 3, 600), "bf16", 1),
    ((2, 8, 2, 5, 3000, 64, 64, 40, 2900), "f32", 8), ((1, 32, 2, 900, 1000, 64, 128, 2, 90), "bf16", 0)],
    ids=["lone", "block", "cluster", "lone-two-rows-a-group"])
def test_the_rule_reaches_each(shape, dtype, share, monkeypatch):
    """Left to itself the rule takes this share: the same bits, which others do not give."""
    monkeypatch.setenv("HILS_Q8_KERNEL", "rows")
    p, h, dev = c8.attend_case(*shape, dtype, dtype, 840)
    O = c8.attend(p, dev)
    same = {}
    for s in range(9):
        monkeypatch.setenv("HILS_Q8_SHARE", str(s))
        same[s] = torch.equal(O.view(torch.uint8), c8.attend(p, dev).view(torch.uint8))
    c8.ok()
    assert same[share]
    assert not all(same.values())
    monkeypatch.delenv("HILS_Q8_SHARE")
    rows = range(0, p.N, max(1, p.N // 23))
    c8.compare(p, h, O, dtype, rows=rows)
    assert np.isfinite(O.float().cpu().numpy()).all()
