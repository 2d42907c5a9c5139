"""The 8-bit cache where the numbers are unusual: what a row gives no weight to does not reach its result, however large the
products with it would be, and a value read back is rounded once, whatever its scale."""
import numpy as np
import pytest
import torch

import cache8_ref as ref
import chunk_wise_hierarchical_hils_b200 as hils
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


def bf16_nearest(x):
    """float64 rounded once to bf16's 8 significant bits (halves to even; subnormals in steps of 2^-133)."""
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e, -125) - 8)
    return np.rint(x / step) * step


def test_read_rounds_once():
    """Scales of 24 bits: scale * value has up to 28 and is rounded to bf16 from all of them.  The scales are chosen so that a
    product lies next to the middle between two bf16 numbers, closer than float32 tells apart."""
    r = np.random.default_rng(620)
    B, Hkv, T, d, C = 1, 2, 1 << 13, 64, 32
    nL = T // C
    data = [r.integers(0, 256, (B, Hkv, T, d), dtype=np.uint8) for _ in range(2)]
    middle = [(2 * r.integers(128, 256, (B, Hkv, nL)) + 1) / r.integers(9, 16, (B, Hkv, nL)) for _ in range(2)]
    scale = [(m * 2.0 ** r.integers(-20, 20, (B, Hkv, nL))).astype(np.float32) for m in middle]
    scale[1][:, :, ::4] *= np.float32(2.0 ** -112)                  # results at and below the smallest normal number
    scale[1][:, :, 1::4] = (r.uniform(1.0, 2.0, scale[1][:, :, 1::4].shape) * 2.0 ** -135).astype(np.float32)
    want = [ref.TABLE[x] * s.astype(np.float64)[:, :, np.arange(T) // C, None] for x, s in zip(data, scale)]
    nan = [np.isnan(w) for w in want]
    once = [bf16_nearest(np.where(n, 0.0, w)) for w, n in zip(want, nan)]
    twice = [torch.from_numpy(np.where(n, 0.0, w).astype(np.float32)).to(torch.bfloat16).double().numpy() for w, n in zip(want, nan)]
    assert all(np.any(a != b) for a, b in zip(once, twice))
    p = hils.problem(B, Hkv, Hkv, 1, T, d, C, 0, 0, hils.HILS_BF16)
    out = [torch.empty((B, Hkv, T, d), dtype=torch.bfloat16, device=c8.DEV) for _ in range(2)]
    dd, sd = [torch.from_numpy(x).to(c8.DEV) for x in data], [torch.from_numpy(x).to(c8.DEV) for x in scale]
    hils.hils_cache_read_q8(p, dd[0], dd[1], sd[0], sd[1], out[0], out[1], 0, T)
    c8.ok()
    for side in range(2):
        got = out[side].double().cpu().numpy()
        assert np.all(np.isnan(got[nan[side]]))
        assert np.array_equal(np.where(nan[side], 0.0, got), once[side])


def test_a_build_without_the_union_kernel_takes_the_rows(monkeypatch):
    """Where the union kernel's build does not have the registers its warps share out, calls that would take it run by rows;
    only a call that asks for it by name fails, and launches nothing."""
    p, h, dev = c8.attend_case(1, 8, 2, 512, 512, 128, 64, 4, 0, "bf16", "bf16", 650)
    out = {}
    for kernel in ("rows", "union", None):
        if kernel:
            monkeypatch.setenv("HILS_Q8_KERNEL", kernel)
        else:
            monkeypatch.delenv("HILS_Q8_KERNEL")
        out[kernel] = c8.attend(p, dev)
    c8.ok()
    same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))   # noqa: E731
    assert same(out[None], out["union"]) and not same(out[None], out["rows"])    # the union's, left to itself
    monkeypatch.setenv("HILS_Q8_UNION_UNFIT", "1")
    O = c8.attend(p, dev)
    c8.ok()
    assert same(O, out["rows"])
    monkeypatch.setenv("HILS_Q8_KERNEL", "union")
    O = torch.full_like(O, 7.0)
    with pytest.raises(hils.HilsError) as e:
        c8.attend(p, dev, O)
    assert e.value.status == hils.HILS_ERR_CUDA
    c8.ok()
    assert torch.all(O == 7.0)
    monkeypatch.delenv("HILS_Q8_UNION_UNFIT")
    assert same(c8.attend(p, dev), out["union"])
    c8.ok()


@pytest.mark.parametrize("N,q0,select", [(1, 450, None), (1, 63, None), (40, 440, None), (100, 400, "heads"), (100, 400, "queries"),
                                         (100, 400, "simt")])
def test_forward_with_anything_behind_the_last_token(N, q0, select, monkeypatch):
    """A cache with room: bytes, scales and landmarks behind the last token's chunk hold anything, NaN among it, and the forward
    gives what it gives with zeros there."""
    if select == "simt":
        monkeypatch.setenv("HILS_PREFILL_KERNEL", select)
    elif select:
        monkeypatch.setenv("HILS_SELECT_KERNEL", select)
    r = np.random.default_rng(630 + N)
    B, H, Hkv, T, d, C, k = 2, 8, 2, 1200, 128, 64, 3
    p, h, dev = c8.attend_case(B, H, Hkv, N, T, d, C, k, q0, "bf16", "bf16", 640 + N)
    nL, used = -(-T // C), (q0 + N - 1) // C + 1
    _, L = c8.rng_rows(r, (B, Hkv, nL, d), "bf16")
    out = []
    for junk in (0.0, float("nan"), float("inf")):
        L[:, :, used:] = junk
        O = torch.full((B, H, N, d), 7.0, dtype=torch.bfloat16, device=c8.DEV)
        ws = torch.empty(hils.hils_forward_q8_workspace_size(p), dtype=torch.uint8, device=c8.DEV)
        hils.hils_forward_q8(p, dev["Q"], dev["K8"], dev["V8"], dev["ks"], dev["vs"], L, O, ws)
        c8.ok()
        out.append(O)
    assert torch.isfinite(out[0]).all()
    for O in out[1:]:
        assert torch.equal(O.view(torch.int16), out[0].view(torch.int16))


@pytest.mark.parametrize("N,kernel,dtype,out", [(1, "rows", "bf16", "bf16"), (100, "rows", "bf16", "bf16"), (100, "union", "bf16", "bf16"),
                                                (1, "rows", "f32", "f32"), (100, "rows", "f32", "f32")])
@pytest.mark.parametrize("v", [1e-40, 2.0 ** -126])
def test_value_scales_below_the_normal_numbers(N, kernel, dtype, out, v, monkeypatch):
    """Results at and below float32's smallest normal number, held to their own steps: besides the usual relative error half a
    step of the result's subnormal numbers, and half a step of float32's for the weight of each slot, times the largest code."""
    monkeypatch.setenv("HILS_Q8_KERNEL", kernel)
    k = 5

    def edit(h, r):
        h["vs"] = np.where(np.isnan(h["vs"]), np.nan, np.float32(v)).astype(np.float32)
    p, h, dev = c8.attend_case(1, 8, 2, N, 400, 128, 64, k, 250, dtype, out, 660 + N, edit=edit)
    O = c8.attend(p, dev)
    c8.ok()
    o, far = O.double().cpu().numpy(), 0.0
    step = {"bf16": 2.0 ** -134, "f32": 2.0 ** -150}[out] + (k + 1) * 448 * 2.0 ** -150
    for g in range(2):
        kd, vd = ref.TABLE[h["K8"][0, g]], ref.TABLE[h["V8"][0, g]]
        for i in range(N):
            ch, sc = np.append(h["sel"][0, g, i], (250 + i) // 64), h["score"][0, 4 * g:4 * g + 4, i].astype(np.float64)
            want, reach, mag = ref.attend_row(h["Q"][0, 4 * g:4 * g + 4, i], kd, vd, h["ks"][0, g].astype(np.float64),
                                              h["vs"][0, g].astype(np.float64), ch, sc, 250 + i, 64, 128 ** -0.5)
            tol = ref.bound(reach, mag, want, out, 128, 64, np.abs(sc[np.isfinite(sc)]).max()) - 1e-37 + step
            assert np.all(np.abs(o[0, 4 * g:4 * g + 4, i] - want) <= tol)
            far = max(far, float(np.max(np.abs(want) / tol)))
    assert far > 20                                         # zeros would not pass
