"""The 8-bit cache on the GPU against the 64-bit reference (cache8_ref): bytes and scales exactly, landmarks and attention
within bounds derived there."""
import math

import numpy as np
import pytest
import torch

import cache8_ref as ref
import chunk_wise_hierarchical_hils_b200 as hils

pytestmark = pytest.mark.gpu

DEV = "cuda"
TD = {"f32": torch.float32, "bf16": torch.bfloat16}
HD = {"f32": hils.HILS_F32, "bf16": hils.HILS_BF16}


def rng_rows(r, shape, dtype, scale=1.0):
    """Normal rows rounded to dtype: (float64 array, device tensor)."""
    t = torch.from_numpy((r.standard_normal(shape) * scale).astype(np.float32)).to(TD[dtype])
    return t.double().numpy(), t.to(DEV)


def empty_cache(B, Hkv, T, d, C, r=None):
    """A cache of arbitrary bytes and scales, as uninitialised memory holds: (data, scale) numpy."""
    r = r or np.random.default_rng(0)
    nL = -(-T // C)
    return r.integers(0, 256, (B, Hkv, T, d), dtype=np.uint8), np.full((B, Hkv, nL), np.nan, np.float32)


def ok():
    assert hils.hils_sync_status() == hils.HILS_OK


def check_append(B, Hkv, T, d, C, dtype, pieces, seed, rows=None):
    r = np.random.default_rng(seed)
    p = hils.problem(B, Hkv, Hkv, 1, T, d, C, 0, 0, HD[dtype])
    state = [empty_cache(B, Hkv, T, d, C, r) for _ in range(2)]
    dev = [(torch.from_numpy(a.copy()).to(DEV), torch.from_numpy(s.copy()).to(DEV)) for a, s in state]
    for t0, t1 in pieces:
        new = []
        for side in range(2):
            x64, xd = rng_rows(r, (B, Hkv, t1 - t0, d), dtype, 10.0 ** r.uniform(-2, 2)) if rows is None else rows(r, t0, t1)
            new.append(xd)
            data, scale = state[side]
            for b in range(B):
                for g in range(Hkv):
                    ref.append(x64[b, g], data[b, g], scale[b, g], t0, C)
        hils.hils_cache_append_q8(p, new[0], new[1], dev[0][0], dev[1][0], dev[0][1], dev[1][1], t0, t1)
    ok()
    for side in range(2):
        got, want = dev[side][0].cpu().numpy(), state[side][0]
        assert np.array_equal(dev[side][1].cpu().numpy(), state[side][1], equal_nan=True)
        same = got == want
        if rows is not None:                               # a NaN keeps no sign
            same |= ((got & 127) == 127) & ((want & 127) == 127)
        assert np.all(same), np.argwhere(~same)[:5]
    return p, state, dev


@pytest.mark.parametrize("B,Hkv,T,d,C,dtype,pieces", [
    (1, 1, 1, 64, 32, "f32", [(0, 1)]),
    (2, 3, 200, 128, 64, "bf16", [(0, 200)]),
    (1, 2, 200, 128, 64, "bf16", [(0, 61), (61, 62), (62, 63), (63, 66), (66, 130), (130, 191)]),
    (2, 1, 333, 64, 32, "f32", [(45, 45 + 177), (222, 223), (223, 333)]),        # starts inside a chunk of old bytes
    (1, 2, 300, 128, 128, "f32", [(0, 1), (1, 127), (127, 129), (129, 300)]),
    (2, 2, 129, 64, 128, "bf16", [(0, 129)]),
    (1, 1, 70, 64, 64, "bf16", [(i, i + 1) for i in range(70)]),
])
def test_append(B, Hkv, T, d, C, dtype, pieces):
    if pieces[0][0]:
        # the chunk the first piece starts in needs a scale of its own: write it first
        pieces = [(pieces[0][0] // C * C, pieces[0][0])] + pieces
    check_append(B, Hkv, T, d, C, dtype, pieces, 300 + T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_special_values(dtype):
    """Infinities and NaN have no say in the scale; zeros, the smallest and the largest numbers."""
    vals = [0.0, -0.0, math.inf, -math.inf, math.nan, 3.3e38, -3.3e38, 1e-40, 1e-38, 448.0, 449.0, 464.0, 480.0, 1.0, 2.0 ** -9,
            2.0 ** -10, 3 * 2.0 ** -11, 17.0, 18.0, 19.0]

    def rows(r, t0, t1):
        x = np.array(vals)[r.integers(0, len(vals), (1, 4, t1 - t0, 64))]
        x[:, 1] = np.where(np.abs(x[:, 1]) < 1e30, x[:, 1], 0.0)          # a kv-head without the largest ones
        x[:, 2] = np.where(np.abs(x[:, 2]) < 1e-30, x[:, 2], math.nan)    # nothing but tiny numbers and NaN
        x[:, 3] = np.where(r.random(x[:, 3].shape) < 0.5, math.inf, math.nan)
        t = torch.from_numpy(x.astype(np.float32)).to(TD[dtype])
        return t.double().numpy(), t.to(DEV)

    check_append(1, 4, 100, 64, 32, dtype, [(0, 40), (40, 41), (41, 100)], 310, rows)


def test_append_token_by_token_equals_at_once():
    """Scales agree, and bytes wherever no value fell below the smallest normal one on the way."""
    r = np.random.default_rng(320)
    x64, xd = rng_rows(r, (1, 2, 96, 128), "bf16")
    p = hils.problem(1, 2, 2, 1, 96, 128, 64, 0, 0, hils.HILS_BF16)
    out = []
    for step in (1, 5, 96):
        a = torch.zeros((1, 2, 96, 128), dtype=torch.uint8, device=DEV)
        s = torch.zeros((1, 2, 2), device=DEV)
        b, z = a.clone(), s.clone()
        for t in range(0, 96, step):
            e = min(t + step, 96)
            piece = xd[:, :, t:e].contiguous()
            hils.hils_cache_append_q8(p, piece, piece, a, b, s, z, t, e)
        ok()
        assert torch.equal(a, b) and torch.equal(s, z)
        out.append((a, s))
    for a, s in out[:2]:
        assert torch.equal(s, out[2][1])
        normal = (out[2][0] & 0x78) != 0
        assert torch.equal(a[normal], out[2][0][normal])


@pytest.mark.parametrize("B,Hkv,T,d,C,dtype,t0,t1", [
    (1, 1, 1, 64, 32, "bf16", 0, 1), (2, 3, 333, 128, 64, "bf16", 0, 333), (1, 2, 333, 64, 32, "f32", 31, 300),
    (2, 1, 700, 128, 128, "f32", 127, 129), (1, 2, 1000, 128, 64, "bf16", 999, 1000), (3, 1, 200, 64, 128, "bf16", 5, 200),
])
def test_read(B, Hkv, T, d, C, dtype, t0, t1):
    r = np.random.default_rng(330 + T)
    nL = -(-T // C)
    data = [r.integers(0, 256, (B, Hkv, T, d), dtype=np.uint8) for _ in range(2)]
    data[0][(data[0] & 127) == 127] = 0x7E
    scale = [np.exp2(r.integers(-100, 100, (B, Hkv, nL))).astype(np.float32) for _ in range(2)]
    if dtype == "f32":
        scale[1] = (scale[1] * np.float32(1.2345)).astype(np.float32)      # any finite scale reads back
    p = hils.problem(B, Hkv, Hkv, 1, T, d, C, 0, 0, HD[dtype])
    out = [torch.full((B, Hkv, t1 - t0, d), 7.0, dtype=TD[dtype], device=DEV) for _ in range(2)]
    dd, sd = [torch.from_numpy(x).to(DEV) for x in data], [torch.from_numpy(x).to(DEV) for x in scale]
    hils.hils_cache_read_q8(p, dd[0], dd[1], sd[0], sd[1], out[0], out[1], t0, t1)
    ok()
    t = np.arange(t0, t1)
    for side in range(2):
        want = ref.TABLE[data[side][:, :, t0:t1]] * scale[side].astype(np.float64)[:, :, t // C, None]
        want = torch.from_numpy(want.astype(np.float32)).to(TD[dtype]).double().numpy()
        assert np.array_equal(out[side].double().cpu().numpy(), want, equal_nan=True)


def make_cache(r, B, Hkv, T, d, C, filled, spread=0.0):
    """A cache written in the first `filled` tokens: bytes, scales (numpy); arbitrary bytes and NaN scales behind."""
    data, scale = empty_cache(B, Hkv, T, d, C, r)
    nb = -(-filled // C)
    x = r.standard_normal((B, Hkv, filled, d))
    level = np.exp2(np.floor(r.uniform(-spread, spread + 1e-9, (B, Hkv, nb))))
    for b in range(B):
        for g in range(Hkv):
            for c in range(nb):
                rows = x[b, g, c * C:(c + 1) * C]
                s = ref.scale_for(np.abs(rows).max())
                data[b, g, c * C:min((c + 1) * C, filled)] = ref.encode(rows / s)
                scale[b, g, c] = s * level[b, g, c]
    return data, scale


@pytest.mark.parametrize("B,Hkv,T,d,C,dtype,c0,c1,end,umul", [
    (1, 1, 1, 64, 32, "f32", 0, 1, 1, 1.0),
    (2, 3, 333, 128, 64, "bf16", 0, 6, 333, 1.0),
    (1, 2, 400, 128, 64, "f32", 2, 4, 197, 1.0),           # the last chunk holds five tokens; stale bytes behind
    (2, 1, 300, 64, 32, "bf16", 1, 8, 250, 6.0),
    (1, 2, 700, 128, 128, "f32", 0, 6, 700, 1.0),
    (1, 1, 700, 64, 128, "bf16", 5, 6, 641, 1.0),
    (16, 8, 256, 128, 64, "bf16", 3, 4, 256, 1.0),
    (1, 2, 520, 128, 32, "f32", 0, 17, 513, 20.0),         # peaked: entropies near zero
    (1, 1, 160, 64, 64, "f32", 0, 3, 160, 1.0),
])
def test_landmarks(B, Hkv, T, d, C, dtype, c0, c1, end, umul):
    r = np.random.default_rng(340 + T + d)
    data, scale = make_cache(r, B, Hkv, T, d, C, end, spread=2.0)
    nL = -(-T // C)
    U64, U = rng_rows(r, (B, Hkv, nL, d), dtype, umul)
    p = hils.problem(B, Hkv, Hkv, 1, T, d, C, 0, 0, HD[dtype])
    L = torch.full((B, Hkv, nL, d), 7.0, dtype=TD[dtype], device=DEV)
    beta = torch.full((B, Hkv, nL), 7.0, device=DEV)
    Kd, sd = torch.from_numpy(data).to(DEV), torch.from_numpy(scale).to(DEV)
    hils.hils_landmarks_q8(p, Kd, sd, U, L, beta, c0, c1, end)
    L2 = torch.empty_like(L)
    hils.hils_landmarks_q8(p, Kd, sd, U, L2, None, c0, c1, end)
    ok()
    assert torch.equal(L2[:, :, c0:c1], L[:, :, c0:c1])
    Lh, bh = L.double().cpu().numpy(), beta.double().cpu().numpy()
    sc = 1.0 / math.sqrt(d)
    for b in range(B):
        for g in range(Hkv):
            for c in range(nL):
                if not c0 <= c < c1:
                    assert np.all(Lh[b, g, c] == 7.0) and bh[b, g, c] == 7.0
                    continue
                k = ref.TABLE[data[b, g, c * C:min((c + 1) * C, end)]] * float(scale[b, g, c])
                wl, wb = ref.landmarks(k, U64[b, g, c], sc)
                # logits within (d + 8) 2^-24 of their magnitudes' sum; the weights move by twice that, the entropy by
                # that times the spread of the logits besides
                mag = float(np.max(np.abs(k) @ np.abs(U64[b, g, c]))) * sc
                e = 2 * (d + 8) * 2.0 ** -24 * mag + (C + 40) * 2.0 ** -24
                tol = e * np.max(np.abs(k)) + ref.half_step(dtype) * np.abs(wl)
                assert np.all(np.abs(Lh[b, g, c] - wl) <= tol)
                assert abs(bh[b, g, c] - wb) <= e * (1 + 2 * mag) + 2.0 ** -22


def make_selection(r, B, Hkv, N, q0, C, k):
    """Random distinct past chunks in random order, -1 behind them; now and then fewer than there are."""
    sel = np.full((B, Hkv, N, k), -1, np.int32)
    for b in range(B):
        for g in range(Hkv):
            for i in range(N):
                ci = (q0 + i) // C
                m = min(k, ci)
                if m and r.random() < 0.1:
                    m = int(r.integers(0, m + 1))
                sel[b, g, i, :m] = r.permutation(ci)[:m]
    return sel


def attend(p, dev, O=None, stream=None):
    B, H, N, d = p.B, p.H, p.N, p.d
    if O is None:
        O = torch.full((B, H, N, d), 7.0, dtype=torch.float32 if p.out_dtype == hils.HILS_F32 else torch.bfloat16, device=DEV)
    ws = torch.empty(max(16, hils.hils_chunk_attend_fuse_q8_workspace_size(p)), dtype=torch.uint8, device=DEV)
    hils.hils_chunk_attend_fuse_q8(p, dev["Q"], dev["K8"], dev["V8"], dev["ks"], dev["vs"], dev["sel"], dev["score"], O, ws,
                                   stream=stream)
    return O


def attend_case(B, H, Hkv, N, T, d, C, k, q0, dtype, out, seed, spread=0.0, qmul=1.0, edit=None):
    r = np.random.default_rng(seed)
    G = H // Hkv
    K8, ks = make_cache(r, B, Hkv, T, d, C, q0 + N)
    V8, vs = make_cache(r, B, Hkv, T, d, C, q0 + N, spread)
    Q64, Q = rng_rows(r, (B, H, N, d), dtype, qmul)
    sel = make_selection(r, B, Hkv, N, q0, C, k)
    score = r.standard_normal((B, H, N, k + 1)).astype(np.float32)
    empty = np.repeat(sel < 0, G, axis=1).reshape(B, H, N, k)
    score[..., :k][empty] = -np.inf
    h = dict(Q=Q64, K8=K8, V8=V8, ks=ks, vs=vs, sel=sel, score=score)
    if edit:
        edit(h, r)
    dev = {n: torch.from_numpy(h[n]).to(DEV) for n in ("K8", "V8", "ks", "vs", "sel", "score")}
    dev["Q"] = Q
    p = hils.problem(B, H, Hkv, N, T, d, C, k, q0, HD[dtype], HD[out])
    return p, h, dev


def compare(p, h, O, out, rows=None):
    B, H, Hkv, N, d, C = p.B, p.H, p.Hkv, p.N, p.d, p.C
    G = H // Hkv
    o = O.double().cpu().numpy()
    assert np.all(np.isfinite(o))
    worst = 0.0
    for b in range(B):
        for g in range(Hkv):
            kd, vd = ref.TABLE[h["K8"][b, g]], ref.TABLE[h["V8"][b, g]]
            for i in (range(N) if rows is None else rows):
                pos = p.q_offset + i
                ch = np.append(h["sel"][b, g, i], pos // C)
                sc = h["score"][b, g * G:(g + 1) * G, i].astype(np.float64)
                want, reach, mag = ref.attend_row(h["Q"][b, g * G:(g + 1) * G, i], kd, vd, h["ks"][b, g].astype(np.float64),
                                                  h["vs"][b, g].astype(np.float64), ch, sc, pos, C, 1.0 / math.sqrt(d))
                fin = np.abs(sc[np.isfinite(sc)])
                tol = ref.bound(reach, mag, want, out, d, C, fin.max() if fin.size else 0.0)
                err = np.abs(o[b, g * G:(g + 1) * G, i] - want)
                assert np.all(err <= tol), (b, g, i, float(np.max(err - tol)), float(np.max(err)), float(np.max(tol)))
                worst = max(worst, float(np.max(err / tol)))
    return worst


SHAPES = [
    # B, H, Hkv, N, T, d, C, k, q0
    (1, 1, 1, 1, 1, 64, 32, 4, 0),                  # one token, no past
    (1, 4, 1, 1, 5, 128, 64, 0, 3),                 # own chunk only
    (2, 8, 2, 1, 1000, 128, 64, 7, 900),            # single token inside a chunk, stale bytes behind
    (1, 16, 1, 1, 4096, 128, 64, 64, 4095),         # 16 heads a group, 65 slots
    (3, 3, 1, 1, 777, 64, 32, 11, 776),             # three heads a group
    (1, 8, 1, 1, 3000, 128, 128, 20, 2900),
    (2, 18, 2, 1, 500, 64, 128, 3, 400),            # nine heads a group
    (16, 32, 8, 1, 640, 128, 64, 8, 639),
    (1, 4, 1, 7, 300, 128, 64, 3, 290),             # a few tokens at once
    (1, 8, 2, 129, 333, 128, 64, 3, 100),           # room behind the last token
    (1, 4, 1, 200, 200, 64, 32, 4, 0),
    (1, 2, 2, 150, 300, 128, 128, 2, 100),
    (1, 16, 1, 70, 256, 128, 64, 2, 150),
    (2, 4, 2, 260, 260, 128, 64, 2, 0),
    (1, 8, 1, 100, 4000, 128, 64, 16, 3890),
    (1, 1, 1, 130, 700, 128, 64, 6, 500),           # one head
    (1, 2, 1, 65, 400, 128, 64, 0, 300),            # own chunk only
    (1, 6, 2, 40, 300, 128, 64, 3, 200),            # three heads a group
]


@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_attend(shape, dtype, out):
    p, h, dev = attend_case(*shape, dtype, out, 350 + sum(shape))
    O = attend(p, dev)
    ok()
    print("worst error / bound %.3g" % compare(p, h, O, out))


UNION_SHAPES = [
    (1, 4, 1, 2, 2, 128, 64, 1, 0),                 # two queries, one chunk
    (1, 4, 1, 33, 500, 128, 64, 3, 190),            # a second block of one query
    (1, 1, 1, 129, 300, 128, 64, 2, 100),           # one head: 128 queries a block
    (1, 2, 1, 200, 4000, 128, 64, 20, 3700),        # many chunks, few of them shared
    (2, 16, 2, 50, 700, 128, 64, 9, 600),           # eight heads a group
    (1, 16, 1, 40, 900, 128, 64, 5, 800),           # sixteen
    (1, 4, 1, 64, 64, 128, 64, 0, 0),               # own chunk only, a lone last pair
    (1, 4, 1, 128, 40000, 128, 64, 37, 39000),      # the longest list of slots that the kernel's shared memory holds, nearly
]


@pytest.mark.parametrize("kernel", ["rows", "union"])
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[3] > 1 and s[5:7] == (128, 64) and s[1] // s[2] in (1, 2, 4, 8, 16)]
                         + UNION_SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_attend_kernels(shape, kernel, monkeypatch):
    """Both kernels of bf16 prefill, whatever the choice between them."""
    monkeypatch.setenv("HILS_Q8_KERNEL", kernel)
    p, h, dev = attend_case(*shape, "bf16", "bf16", 500 + sum(shape))
    O = attend(p, dev)
    O2 = attend(p, dev)
    ok()
    assert torch.equal(O.view(torch.int16), O2.view(torch.int16))
    compare(p, h, O, "bf16")


def test_attend_union_on_shared_selections(monkeypatch):
    """Neighbouring queries that keep the same chunks (the union is short) and rows with nothing selected."""
    monkeypatch.setenv("HILS_Q8_KERNEL", "union")

    def edit(h, r):
        h["sel"][:] = h["sel"][:, :, :1]                   # the first query's chunks for all
        h["sel"][:, :, 5:9] = -1
    p, h, dev = attend_case(1, 8, 2, 100, 2000, 128, 64, 16, 1880, "bf16", "bf16", 520, edit=edit)
    O = attend(p, dev)
    ok()
    compare(p, h, O, "bf16")


@pytest.mark.parametrize("kernel", ["rows", "union"])
def test_attend_smallest_and_largest_scales(kernel, monkeypatch):
    """Value scales down to float32's subnormals and up to 2^119, in different kv-heads."""
    monkeypatch.setenv("HILS_Q8_KERNEL", kernel)

    def edit(h, r):
        for g, v in enumerate((1e-40, 2.0 ** -100, 2.0 ** 119)):
            h["vs"][:, g] = np.where(np.isnan(h["vs"][:, g]), np.nan, np.float32(v))
    p, h, dev = attend_case(1, 12, 3, 100, 400, 128, 64, 5, 250, "bf16", "bf16", 535, edit=edit)
    O = attend(p, dev)
    ok()
    compare(p, h, O, "bf16")


@pytest.mark.parametrize("kernel", ["rows", "union"])
def test_attend_wide_scales_kernels(kernel, monkeypatch):
    monkeypatch.setenv("HILS_Q8_KERNEL", kernel)
    p, h, dev = attend_case(1, 8, 2, 140, 400, 128, 64, 5, 200, "bf16", "bf16", 530, spread=60.0)
    O = attend(p, dev)
    ok()
    compare(p, h, O, "bf16")


def test_attend_zero_queries_and_zero_scales():
    """Queries of zeros see every key alike; chunks of scale zero (keys or values) are chunks of zeros."""
    def edit(h, r):
        h["ks"][:, :, ::2] = np.where(np.isnan(h["ks"][:, :, ::2]), np.nan, 0.0)
        h["vs"][:, :, 1::3] = np.where(np.isnan(h["vs"][:, :, 1::3]), np.nan, 0.0)
    for N, q0 in ((1, 700), (96, 600)):
        p, h, dev = attend_case(1, 8, 2, N, 800, 128, 64, 6, q0, "bf16", "bf16", 540 + N, edit=edit)
        h["Q"][:, 1::2] = 0.0
        dev["Q"][:, 1::2] = 0
        O = attend(p, dev)
        ok()
        compare(p, h, O, "bf16")


@pytest.mark.parametrize("shape,dtype,rows", [
    ((1, 2, 2, 1003, 1024, 64, 32, 4, 0), "f32", range(0, 1003, 41)),        # rows enough for a warp each
    ((4, 32, 8, 3, 2000, 128, 64, 12, 1990), "bf16", None),                   # teams of one block
    ((2, 8, 2, 5, 3000, 64, 64, 40, 2900), "f32", None),                      # teams of several
], ids=["lone", "block", "cluster"])
def test_attend_shares_of_rows(shape, dtype, rows):
    p, h, dev = attend_case(*shape, dtype, dtype, 550 + sum(shape))
    O = attend(p, dev)
    ok()
    compare(p, h, O, dtype, rows=rows)


def test_a_cache_beyond_four_gigabytes():
    """Offsets past 32 bits: the last tokens of a 4M-token cache of eight kv-heads (4.3 GB a side)."""
    B, H, Hkv, T, d, C, slots = 1, 16, 8, 1 << 22, 128, 64, 5
    r = np.random.default_rng(560)
    nL = T // C
    K8 = torch.zeros((B, Hkv, T, d), dtype=torch.uint8, device=DEV)
    V8 = torch.zeros_like(K8)
    ks, vs = torch.zeros((B, Hkv, nL), device=DEV), torch.zeros((B, Hkv, nL), device=DEV)
    t0 = T - 5 * C - 17
    x64, x = zip(*(rng_rows(r, (B, Hkv, T - t0, d), "bf16") for _ in range(2)))
    p = hils.problem(B, H, Hkv, 1, T, d, C, slots, T - 1, hils.HILS_BF16, hils.HILS_BF16)
    hils.hils_cache_append_q8(p, x[0][:, :, :17].contiguous(), x[1][:, :, :17].contiguous(), K8, V8, ks, vs, t0, t0 + 17)
    hils.hils_cache_append_q8(p, x[0][:, :, 17:].contiguous(), x[1][:, :, 17:].contiguous(), K8, V8, ks, vs, t0 + 17, T)
    back = [torch.empty_like(x[0]) for _ in range(2)]
    hils.hils_cache_read_q8(p, K8, V8, ks, vs, back[0], back[1], t0, T)
    U64, U = rng_rows(r, (B, Hkv, nL, d), "bf16")
    L = torch.zeros((B, Hkv, nL, d), dtype=torch.bfloat16, device=DEV)
    hils.hils_landmarks_q8(p, K8, ks, U, L, None, nL - 5, nL)
    ok()
    assert not K8[:, :, :t0].any() and not V8[:, :, :t0].any()
    # the last kv-heads' tails on the host
    tail = 6 * C
    base = T - tail
    for g in (0, Hkv - 1):
        data, scale = np.zeros((tail, d), np.uint8), np.zeros(6, np.float32)
        ref.append(x64[0][0, g, :17], data, scale, t0 - base, C)
        ref.append(x64[0][0, g, 17:], data, scale, t0 + 17 - base, C)
        assert np.array_equal(K8[0, g, base:].cpu().numpy(), data)
        assert np.array_equal(ks[0, g, -6:].cpu().numpy(), scale)
        val = ref.TABLE[data] * scale.astype(np.float64)[np.arange(tail) // C, None]
        got = back[0][0, g].double().cpu().numpy()
        assert np.array_equal(got, val[t0 - base:])
        for c in (1, 5):
            k, u = val[c * C:(c + 1) * C], U64[0, g, nL - 6 + c]
            want, _ = ref.landmarks(k, u, 1.0 / math.sqrt(d))
            e = 2 * (d + 8) * 2.0 ** -24 * np.max(np.abs(k) @ np.abs(u)) / math.sqrt(d) + (C + 40) * 2.0 ** -24
            tol = e * np.max(np.abs(k)) + ref.half_step("bf16") * np.abs(want)
            assert np.all(np.abs(L[0, g, nL - 6 + c].double().cpu().numpy() - want) <= tol)
    # a query that keeps the five chunks before its own
    Q64, Q = rng_rows(r, (B, H, 1, d), "bf16")
    sel = torch.arange(nL - 6, nL - 1, dtype=torch.int32, device=DEV).view(1, 1, 1, slots).expand(B, Hkv, 1, slots).contiguous()
    score = torch.zeros((B, H, 1, slots + 1), device=DEV)
    O = attend(p, dict(Q=Q, K8=K8, V8=V8, ks=ks, vs=vs, sel=sel, score=score))
    ok()
    h = dict(Q=Q64, K8=K8[:, :, base:].cpu().numpy(), V8=V8[:, :, base:].cpu().numpy(), ks=ks[:, :, -6:].cpu().numpy(),
             vs=vs[:, :, -6:].cpu().numpy(), sel=sel.cpu().numpy() - (nL - 6), score=score.cpu().numpy())
    pt = hils.problem(B, H, Hkv, 1, tail, d, C, slots, tail - 1, hils.HILS_BF16, hils.HILS_BF16)
    compare(pt, h, O, "bf16")


def test_a_stalled_prefill_reports_a_timeout(monkeypatch):
    """The bounded waits of the tensor-core kernel: a wait that nothing ends expires, the status tells, the next call is right."""
    monkeypatch.setenv("HILS_Q8_KERNEL", "union")
    p, h, dev = attend_case(1, 8, 2, 200, 600, 128, 64, 4, 400, "bf16", "bf16", 570)
    try:
        hils.hils_set_wait_limit(2_000_000)                 # 2 ms
        hils.hils_debug_inject_stall(1)
        attend(p, dev)
        assert hils.hils_sync_status() == hils.HILS_ERR_TIMEOUT
    finally:
        hils.hils_debug_inject_stall(0)
        hils.hils_set_wait_limit(0)
    O = attend(p, dev)
    ok()
    compare(p, h, O, "bf16", rows=range(0, 200, 7))


@pytest.mark.parametrize("shape", [(1, 4, 1, 1, 1000, 128, 64, 9, 999), (1, 8, 2, 140, 400, 128, 64, 5, 200),
                                   (1, 4, 2, 30, 300, 64, 32, 5, 200)], ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32")])
def test_attend_wide_scales(shape, dtype, out):
    """Value scales from 2^-60 to 2^60 of one another, queries of one row far apart in size."""
    def edit(h, r):
        pass
    p, h, dev = attend_case(*shape, dtype, out, 360 + sum(shape), spread=60.0, edit=edit)
    O = attend(p, dev)
    ok()
    compare(p, h, O, out)


@pytest.mark.parametrize("qexp", [-60, -20, 40])
@pytest.mark.parametrize("N", [1, 100])
def test_attend_wide_queries(qexp, N):
    """Queries and key scales far from one, their products ordinary."""
    def edit(h, r):
        h["ks"] = (h["ks"] * np.float32(2.0 ** -qexp)).astype(np.float32)
    p, h, dev = attend_case(1, 8, 2, N, 400, 128, 64, 4, 300, "bf16", "bf16", 370 + N, qmul=2.0 ** qexp, edit=edit)
    O = attend(p, dev)
    ok()
    compare(p, h, O, "bf16")


@pytest.mark.parametrize("N", [1, 40, 140])
@pytest.mark.parametrize("dtype,out", [("bf16", "bf16"), ("f32", "f32")])
def test_attend_empty_slots_and_masked_scores(N, dtype, out):
    """Slots of -1 hold any score; a slot of score -inf has no weight; a row of none is zero."""
    def edit(h, r):
        B, Hkv, N_, k = h["sel"].shape
        H = h["score"].shape[1]
        empty = np.repeat(h["sel"] < 0, H // Hkv, axis=1).reshape(B, H, N_, k)
        h["sel"][:, :, ::3, 1] = -1
        empty = np.repeat(h["sel"] < 0, H // Hkv, axis=1).reshape(B, H, N_, k)
        junk = np.array([np.nan, np.inf, -np.inf, 3.0e38], np.float32)
        h["score"][..., :k][empty] = junk[r.integers(0, 4, int(empty.sum()))]
        h["score"][:, 0, :, 0] = -np.inf                   # one head of a group without its first slot
        h["score"][:, 1, ::2, k] = -np.inf                 # the own chunk without weight
        h["score"][:, 2, ::5, :] = -np.inf                 # nothing left
    p, h, dev = attend_case(1, 8, 2, N, 600, 128, 64, 5, 450, dtype, out, 380 + N, edit=edit)
    O = attend(p, dev)
    ok()
    assert torch.all(O[:, 2, ::5] == 0)
    compare(p, h, O, out)


@pytest.mark.parametrize("N,kernel", [(1, "rows"), (40, "rows"), (140, "rows"), (140, "union")])
def test_attend_entries_outside_the_past(N, kernel, monkeypatch):
    """Entries that name no past chunk (the own one, later ones, far outside, negative) are empty slots."""
    monkeypatch.setenv("HILS_Q8_KERNEL", kernel)

    def edit(h, r):
        own = (450 + np.arange(N)) // 64
        bad = np.stack([own, own + 1, np.full(N, 2 ** 31 - 1), np.full(N, -2 ** 31), np.full(N, 10 ** 6), np.full(N, -2)], -1)
        h["given"] = h["sel"].copy()
        at = r.integers(0, 6, (h["sel"].shape[1], N))
        for g in range(h["sel"].shape[1]):
            h["given"][0, g, :, 2] = bad[np.arange(N), at[g]]
        h["sel"][:, :, :, 2] = -1
        h["score"][:, :, :, 2] = 1.0
    p, h, dev = attend_case(1, 8, 2, N, 600, 128, 64, 5, 450, "bf16", "bf16", 385 + N, edit=edit)
    dev["sel"] = torch.from_numpy(h["given"]).to(DEV)
    O = attend(p, dev)
    ok()
    compare(p, h, O, "bf16")


@pytest.mark.parametrize("kernel", ["rows", "union"])
def test_attend_a_chunk_named_twice_harms_no_other_row(kernel, monkeypatch):
    monkeypatch.setenv("HILS_Q8_KERNEL", kernel)
    N = 140

    def edit(h, r):
        h["sel"][:, :, ::2, 3] = h["sel"][:, :, ::2, 0]
        h["sel"][:, :, ::6] = h["sel"][:, :, ::6, :1]       # in every slot
    p, h, dev = attend_case(1, 8, 2, N, 600, 128, 64, 5, 450, "bf16", "bf16", 527, edit=edit)
    O = attend(p, dev)
    ok()
    compare(p, h, O, "bf16", rows=range(1, N, 2))


@pytest.mark.parametrize("N", [1, 64])
def test_attend_extreme_scores(N):
    """Scores at the type's lowest and highest values."""
    def edit(h, r):
        h["score"][:, :, :, 0] = np.float32(-3.4028235e38)
        h["score"][:, 1, :, 1] = np.float32(3.0e38)
    p, h, dev = attend_case(1, 4, 1, N, 600, 128, 64, 5, 450, "bf16", "bf16", 390 + N, edit=edit)
    O = attend(p, dev)
    ok()
    G = p.H
    h["score"][:, :, :, 0] = -np.inf                        # the same weights, without 1e38 in the bound
    h["score"][:, 1, :, :] = np.where(np.arange(6) == 1, 0.0, -np.inf)
    sel0 = h["sel"][..., 1] < 0
    keep = [i for i in range(N) if not sel0[0, 0, i]]
    compare(p, h, O, "bf16", rows=keep)
    assert G == 4


def test_attend_is_repeatable_and_leaves_its_inputs():
    p, h, dev = attend_case(1, 8, 2, 150, 500, 128, 64, 6, 340, "bf16", "bf16", 400)
    before = {n: t.clone() for n, t in dev.items()}
    a = attend(p, dev)
    b = attend(p, dev)
    ok()
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    for n, t in dev.items():
        assert torch.equal(t.view(torch.uint8), before[n].view(torch.uint8)), n


@pytest.mark.parametrize("N,q0", [(1, 700), (130, 500)])
def test_attend_on_other_streams_and_in_graphs(N, q0):
    """Two streams with workspaces of their own at once, and a captured call replayed on new data."""
    cases = [attend_case(2, 8, 2, N, 800, 128, 64, 6, q0, "bf16", "bf16", 410 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(3):
        for i, (p, _, dev) in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                outs[i].append(attend(p, dev))
    torch.cuda.synchronize()
    for i, (p, h, dev) in enumerate(cases):
        assert all(torch.equal(o.view(torch.int16), outs[i][0].view(torch.int16)) for o in outs[i])
        compare(p, h, outs[i][0], "bf16", rows=range(0, N, 9))
    p, h, dev = cases[0]
    ws = torch.empty(max(16, hils.hils_chunk_attend_fuse_q8_workspace_size(p)), dtype=torch.uint8, device=DEV)
    O = torch.empty((2, 8, N, 128), dtype=torch.bfloat16, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        hils.hils_chunk_attend_fuse_q8(p, dev["Q"], dev["K8"], dev["V8"], dev["ks"], dev["vs"], dev["sel"], dev["score"], O, ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(O.view(torch.int16), outs[0][0].view(torch.int16))
    for n, t in dev.items():
        t.copy_(cases[1][2][n])
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(O.view(torch.int16), outs[1][0].view(torch.int16))
    del g


def test_cache_calls_in_a_graph_and_on_a_stream():
    """append, read and landmarks captured together and replayed on new rows."""
    r = np.random.default_rng(420)
    B, Hkv, T, d, C, t0, t1 = 2, 2, 256, 128, 64, 0, 130
    p = hils.problem(B, Hkv, Hkv, 1, T, d, C, 0, 0, hils.HILS_BF16)
    x64, x = rng_rows(r, (B, Hkv, t1, d), "bf16")
    _, U = rng_rows(r, (B, Hkv, 4, d), "bf16")
    K8 = torch.zeros((B, Hkv, T, d), dtype=torch.uint8, device=DEV)
    V8, ks = torch.zeros_like(K8), torch.zeros((B, Hkv, 4), device=DEV)
    vs, back, back2 = torch.zeros_like(ks), torch.empty_like(x), torch.empty_like(x)
    L = torch.zeros((B, Hkv, 4, d), dtype=torch.bfloat16, device=DEV)

    def calls():
        hils.hils_cache_append_q8(p, x, x, K8, V8, ks, vs, t0, t1)
        hils.hils_cache_read_q8(p, K8, V8, ks, vs, back, back2, t0, t1)
        hils.hils_landmarks_q8(p, K8, ks, U, L, None, 0, None, t1)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        calls()
    torch.cuda.synchronize()
    first = (back.clone(), L.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    back.zero_(); L.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(back, first[0]) and torch.equal(L, first[1]) and torch.equal(back, back2)
    # a value is off by at most half a step of its own, or of the smallest normal one
    step = np.maximum(np.abs(x64) * 2.0 ** -4, np.repeat(ks.double().cpu().numpy()[:, :, :3], C, 2)[:, :, :t1, None] * 2.0 ** -10)
    assert np.all(np.abs(back.double().cpu().numpy() - x64) <= step)
    x.neg_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(back, -first[0])
    del g


def test_a_sequence_served_from_the_cache():
    """A prompt is written, its landmarks made, its queries answered; then tokens one by one: each writes its row, completes a
    chunk's landmark where it does, and attends.  Selection is the library's own; attention is checked on it."""
    r = np.random.default_rng(430)
    B, H, Hkv, d, C, k, T, n0, steps = 2, 8, 2, 128, 64, 3, 512, 300, 40
    x = {s: rng_rows(r, (B, Hkv, n0 + steps, d), "bf16")[1] for s in "KV"}
    Qall = rng_rows(r, (B, H, n0 + steps, d), "bf16")[1]
    nL = T // C
    U = rng_rows(r, (B, Hkv, nL, d), "bf16")[1]
    K8 = torch.randint(0, 256, (B, Hkv, T, d), dtype=torch.uint8, device=DEV)
    V8 = torch.randint(0, 256, (B, Hkv, T, d), dtype=torch.uint8, device=DEV)
    ks, vs = torch.full((B, Hkv, nL), math.nan, device=DEV), torch.full((B, Hkv, nL), math.nan, device=DEV)
    L = torch.zeros((B, Hkv, nL, d), dtype=torch.bfloat16, device=DEV)

    def step(t0, t1):
        N = t1 - t0
        p = hils.problem(B, H, Hkv, N, T, d, C, k, t0, hils.HILS_BF16, hils.HILS_BF16)
        hils.hils_cache_append_q8(p, x["K"][:, :, t0:t1].contiguous(), x["V"][:, :, t0:t1].contiguous(), K8, V8, ks, vs, t0, t1)
        hils.hils_landmarks_q8(p, K8, ks, U, L, None, t0 // C, -(-t1 // C), t1)
        Q = Qall[:, :, t0:t1].contiguous()
        O = torch.empty((B, H, N, d), dtype=torch.bfloat16, device=DEV)
        ws = torch.empty(hils.hils_forward_q8_workspace_size(p), dtype=torch.uint8, device=DEV)
        hils.hils_forward_q8(p, Q, K8, V8, ks, vs, L, O, ws)
        sel = torch.empty((B, Hkv, N, k), dtype=torch.int32, device=DEV)
        score = torch.empty((B, H, N, k + 1), device=DEV)
        w2 = torch.empty(max(16, hils.hils_score_select_workspace_size(p)), dtype=torch.uint8, device=DEV)
        hils.hils_score_select(p, Q, L, sel, score, w2)
        dev = dict(Q=Q, K8=K8, V8=V8, ks=ks, vs=vs, sel=sel, score=score)
        O2 = attend(p, dev)
        ok()
        assert torch.equal(O.view(torch.int16), O2.view(torch.int16))
        h = {n: t.cpu().numpy() for n, t in dev.items() if n != "Q"}
        h["Q"] = Q.double().cpu().numpy()
        compare(p, h, O, "bf16", rows=range(0, N, 17))
        return O

    step(0, n0)
    for t in range(n0, n0 + steps):
        step(t, t + 1)
    # and near what the same sequence gives on the bf16 cache with the same selection: keys and values are within 2^-4
    t = n0 + steps - 1
    p = hils.problem(B, H, Hkv, 1, t + 1, d, C, k, t, hils.HILS_BF16, hils.HILS_F32)
    Q = Qall[:, :, t:].contiguous()
    back = [torch.empty((B, Hkv, t + 1, d), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    hils.hils_cache_read_q8(hils.problem(B, H, Hkv, 1, T, d, C, k, t, hils.HILS_BF16), K8, V8, ks, vs, back[0], back[1], 0, t + 1)
    Lt = L[:, :, :-(-(t + 1) // C)].contiguous()
    sel = torch.empty((B, Hkv, 1, k), dtype=torch.int32, device=DEV)
    score = torch.empty((B, H, 1, k + 1), device=DEV)
    ws = torch.empty(max(16, hils.hils_score_select_workspace_size(p)), dtype=torch.uint8, device=DEV)
    hils.hils_score_select(p, Q, Lt, sel, score, ws)
    O = torch.empty((B, H, 1, d), device=DEV)
    ws = torch.empty(max(16, hils.hils_chunk_attend_fuse_workspace_size(p)), dtype=torch.uint8, device=DEV)
    hils.hils_chunk_attend_fuse(p, Q, back[0], back[1], sel, score, O, ws)
    p8 = hils.problem(B, H, Hkv, 1, T, d, C, k, t, hils.HILS_BF16, hils.HILS_F32)
    O8 = attend(p8, dict(Q=Q, K8=K8, V8=V8, ks=ks, vs=vs, sel=sel, score=score))
    ok()
    # the same values through both paths: each within the library's bf16 attention bound of the formula
    assert (O - O8).abs().max().item() <= 1e-2


def test_attend_with_a_window_selection():
    """The window's selection (k' = k + window - 1 slots) feeds the 8-bit attention like any other."""
    r = np.random.default_rng(440)
    B, H, Hkv, N, T, d, C, k, wc, q0 = 1, 8, 2, 90, 512, 128, 64, 2, 3, 400
    p = hils.problem(B, H, Hkv, N, T, d, C, k, q0, hils.HILS_BF16, hils.HILS_BF16)
    pk = hils.problem(B, H, Hkv, N, T, d, C, k + wc - 1, q0, hils.HILS_BF16, hils.HILS_BF16)
    _, h, dev = attend_case(B, H, Hkv, N, T, d, C, k + wc - 1, q0, "bf16", "bf16", 441)
    _, L = rng_rows(r, (B, Hkv, T // C, d), "bf16")
    hils.hils_score_select_window(p, wc, None, dev["Q"], L, dev["sel"], dev["score"])
    O = attend(pk, dev)
    ok()
    h["sel"], h["score"] = dev["sel"].cpu().numpy(), dev["score"].cpu().numpy()
    compare(pk, h, O, "bf16", rows=range(0, N, 7))


def test_a_checked_selection_is_refused(monkeypatch):
    p, h, dev = attend_case(1, 4, 2, 5, 300, 128, 64, 3, 250, "bf16", "bf16", 450)
    monkeypatch.setenv("HILS_CHECK_SELECTION", "1")
    attend(p, dev)
    dev["sel"][0, 0, 2, 0] = 4                              # the query's own chunk or later: not a past chunk
    with pytest.raises(hils.HilsError) as e:
        attend(p, dev)
    assert e.value.status == hils.HILS_ERR_INVALID_ARG
