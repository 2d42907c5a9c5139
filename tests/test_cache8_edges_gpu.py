"""The 8-bit cache's attention where a weight is zero and the numbers behind it are not: what a row gives no weight to must
not reach its result, however large the products with it would be."""
import numpy as np
import pytest
import torch

import test_cache8_gpu as c8

pytestmark = pytest.mark.gpu


def far_apart(h, dev, big):
    """Queries of the rows `big` [B,H,N] times 2^80, of all others times 2^-80 (both exact)."""
    f = np.where(big, 2.0 ** 80, 2.0 ** -80)
    h["Q"] *= f[..., None]
    dev["Q"] = torch.from_numpy(h["Q"].astype(np.float32)).to(dev["Q"].dtype).to(c8.DEV)


def scale_keys(h):
    """Even chunks' key scales times 2^80, odd ones' times 2^-80."""
    c = np.arange(h["ks"].shape[-1])
    h["ks"] = (h["ks"] * np.where(c % 2 == 0, 2.0 ** 80, 2.0 ** -80)).astype(np.float32)


@pytest.mark.parametrize("kernel", ["rows", "union"])
def test_queries_far_apart_with_chunks_of_their_own(kernel, monkeypatch):
    """Neighbouring queries 2^160 apart whose chunks' keys make up for it: each one's products with its own chunks are
    ordinary, those with the others' chunks beyond float32.  The own chunk has no weight."""
    monkeypatch.setenv("HILS_Q8_KERNEL", kernel)
    N = 100

    def edit(h, r):
        scale_keys(h)
        for i in range(N):
            for g in range(2):
                past = np.arange(i % 2, 7, 2)                       # even queries take even chunks, odd ones odd chunks
                h["sel"][0, g, i] = r.permutation(past)[:3]
        h["score"][:] = r.standard_normal(h["score"].shape)
        h["score"][..., 3] = -np.inf
    p, h, dev = c8.attend_case(1, 8, 2, N, 600, 128, 64, 3, 450, "bf16", "bf16", 600, edit=edit)
    far_apart(h, dev, np.broadcast_to(np.arange(N) % 2 == 1, (1, 8, N)))
    O = c8.attend(p, dev)
    c8.ok()
    c8.compare(p, h, O, "bf16")


@pytest.mark.parametrize("N,kernel,dtype,out", [(1, "rows", "bf16", "bf16"), (1, "rows", "f32", "f32"), (100, "rows", "bf16", "bf16"),
                                                (100, "union", "bf16", "bf16"), (100, "rows", "f32", "f32"),
                                                (100, "rows", "bf16", "f32")])
def test_heads_far_apart_with_slots_of_their_own(N, kernel, dtype, out, monkeypatch):
    """Heads of a group 2^160 apart, each with weight only in the slots whose keys make up for it."""
    monkeypatch.setenv("HILS_Q8_KERNEL", kernel)

    def edit(h, r):
        scale_keys(h)
        h["sel"][:] = np.stack([r.permutation(7)[:5] for _ in range(2 * N)]).reshape(1, 2, N, 5)
        h["score"][:] = r.standard_normal(h["score"].shape)
        odd_chunk = np.repeat(h["sel"] % 2, 4, axis=1)              # [1,8,N,5]
        odd_head = np.arange(8)[None, :, None, None] % 2
        h["score"][..., :5][odd_chunk != odd_head] = -np.inf
        h["score"][..., 5] = -np.inf
    p, h, dev = c8.attend_case(1, 8, 2, N, 600, 128, 64, 5, 450, dtype, out, 610 + N, edit=edit)
    far_apart(h, dev, np.broadcast_to((np.arange(8) % 2 == 1)[None, :, None], (1, 8, N)))
    O = c8.attend(p, dev)
    c8.ok()
    c8.compare(p, h, O, out)
