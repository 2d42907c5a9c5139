"""How the 8-bit cache's kernels round queries and weights: what the pieces lose, pinned on the CPU, and whole results on the
GPU held to the error those losses add up to.

A bound on every element has to assume that all roundings of a row of 128 products agree; an error of a tenth of it is already
a wrong kernel.  So these checks take the root mean square of the error over a result, relative to the result's own, where
independent roundings add as their squares do."""
import math

import numpy as np
import pytest
import torch

import cache8_ref as ref
import chunk_wise_hierarchical_hils_b200 as hils
import test_cache8_gpu as c8


# ---- the pieces ----------------------------------------------------------------------------------------------------------

def f16(x):
    return np.asarray(x, np.float64).astype(np.float16).astype(np.float64)


def e4m3(x):
    return ref.TABLE[ref.encode(np.asarray(x, np.float64))]


def scaled(q, top):
    """Rows times the power of two that takes their largest magnitude to [2^top, 2^(top + 1)), and that power."""
    f = np.exp2(top + 1 - np.frexp(np.max(np.abs(q), -1, keepdims=True))[1])
    return q * f, f


def pieces(x, rnd, n):
    """x as the sum of n pieces rounded by rnd."""
    s = np.zeros_like(x)
    for _ in range(n):
        s = s + rnd(x - s)
    return s


def query(q, kernel, n=None):
    """A query row as the kernels take it: `rows` in f16 (two pieces of a float32 one), `union` in two e4m3 pieces."""
    x, f = scaled(q, 7 if kernel == "union" else 14)
    return pieces(x, e4m3 if kernel == "union" else f16, n or 2) / f


def test_what_a_query_loses_in_two_e4m3_pieces():
    """Every bf16 number against the smallest and largest bf16 number its row's largest can be in a binade."""
    small = (128 + np.arange(128)) / 128.0
    for top in (1.0, 255 / 128.0):
        for e in range(0, 20):
            q = np.stack(np.broadcast_arrays(small * 2.0 ** -e, top), -1)
            q = q[q[:, 0] <= top]
            loss = np.abs(query(q, "union") - q)[:, 0]
            assert np.all(loss <= 2.0 ** -17 * top) and np.all(loss[q[:, 0] >= 2.0 ** -9 * top] == 0.0)
    q = np.array([[0.125 + 2.0 ** -10, 128.0]]) / 128                # above 2^-10 of the largest, and loses 2^-17 of it
    assert q[0, 0] > 2.0 ** -10 and np.abs(query(q, "union") - q)[0, 0] == 2.0 ** -17


def test_what_a_query_loses_in_f16():
    small = (128 + np.arange(128)) / 128.0
    for top in (1.0, 255 / 128.0):
        for e in range(0, 45):
            q = np.stack(np.broadcast_arrays(small * 2.0 ** -e, top), -1)
            q = q[q[:, 0] <= top]
            loss = np.abs(query(q, "rows", 1) - q)[:, 0]
            assert np.all(loss <= 2.0 ** -39 * top) and np.all(loss[q[:, 0] >= 2.0 ** -31 * top] == 0.0)
    r = np.random.default_rng(700)
    q = (r.standard_normal((1000, 64)) * 2.0 ** r.integers(-45, 1, (1000, 64))).astype(np.float32).astype(np.float64)
    big = np.max(np.abs(q), -1, keepdims=True)
    assert np.all(np.abs(query(q, "rows") - q) <= np.maximum(2.0 ** -22 * np.abs(q), 2.0 ** -39 * big))


def test_what_a_weight_loses_in_f16():
    r = np.random.default_rng(701)
    x = r.uniform(0.5, 1.0, 100000) * 2.0 ** r.integers(-27, 15, 100000)
    for n, rel in ((1, 2.0 ** -11), (2, 2.0 ** -22)):
        loss = np.abs(pieces(x, f16, n) - x)
        assert np.all(loss <= np.maximum(rel * x, 2.0 ** -25))
    assert np.max(np.abs(f16(x) - x) / x) > 0.9 * 2.0 ** -11


# ---- whole results -------------------------------------------------------------------------------------------------------

def host_case(B, H, Hkv, N, T, d, C, k, q0, dtype, out, seed, edit=None):
    """Inputs as c8.attend_case makes them, on the host only: (problem, arrays)."""
    r = np.random.default_rng(seed)
    K8, ks = c8.make_cache(r, B, Hkv, T, d, C, q0 + N)
    V8, vs = c8.make_cache(r, B, Hkv, T, d, C, q0 + N)
    Q = torch.from_numpy(r.standard_normal((B, H, N, d)).astype(np.float32)).to(c8.TD[dtype]).double().numpy()
    sel = c8.make_selection(r, B, Hkv, N, q0, C, k)
    score = r.standard_normal((B, H, N, k + 1)).astype(np.float32)
    score[..., :k][np.repeat(sel < 0, H // Hkv, axis=1).reshape(B, H, N, k)] = -np.inf
    h = dict(Q=Q, K8=K8, V8=V8, ks=ks, vs=vs, sel=sel, score=score)
    if edit:
        edit(h, r)
    return hils.problem(B, H, Hkv, N, T, d, C, k, q0, c8.HD[dtype], c8.HD[out]), h


def on_device(p, h):
    dev = {n: torch.from_numpy(h[n]).to(c8.DEV) for n in ("K8", "V8", "ks", "vs", "sel", "score")}
    dev["Q"] = torch.from_numpy(h["Q"].astype(np.float32)).to(torch.float32 if p.in_dtype == hils.HILS_F32 else torch.bfloat16).to(c8.DEV)
    return dev


def compute(p, h, rows=None, q_as=lambda q: q, p_as=lambda x: x, add=lambda a, b: a + b):
    """The formula in 64 bits [B,H,rows,d]; q_as and p_as stand in for a kernel's rounding of query rows and of weights over
    the row's largest, `add` for how its accumulator takes the products of 16 keys."""
    G, C = p.H // p.Hkv, p.C
    rows = range(p.N) if rows is None else rows
    O = np.zeros((p.B, p.H, len(rows), p.d))
    for b in range(p.B):
        for g in range(p.Hkv):
            for n, i in enumerate(rows):
                pos = p.q_offset + i
                ch = np.append(h["sel"][b, g, i], pos // C)
                q = q_as(h["Q"][b, g * G:(g + 1) * G, i])
                s = np.where(ch < 0, -np.inf, h["score"][b, g * G:(g + 1) * G, i].astype(np.float64))
                w = np.exp(s - s.max(-1, keepdims=True))
                w = w / w.sum(-1, keepdims=True) * np.where(ch < 0, 0.0, h["vs"][b, g][np.maximum(ch, 0)])
                top = w.max(-1, keepdims=True) * 2.0 ** -14
                acc = np.zeros((G, p.d))
                for j, c in enumerate(ch):
                    if c < 0:
                        continue
                    t = slice(c * C, min((c + 1) * C, pos + 1))
                    x = q @ (ref.TABLE[h["K8"][b, g, t]] * float(h["ks"][b, g, c])).T / math.sqrt(p.d)
                    e = np.exp(x - x.max(-1, keepdims=True))
                    e = p_as(e / e.sum(-1, keepdims=True) * w[:, j:j + 1] / top)
                    v = ref.TABLE[h["V8"][b, g, t]]
                    for m in range(0, len(v), 16):
                        acc = add(acc, e[:, m:m + 16] @ v[m:m + 16])
                O[b, g * G:(g + 1) * G, n] = acc * top
    return O


def rms_error(o, want):
    return math.sqrt(np.mean((o - want) ** 2) / np.mean(want ** 2))


def wide_rows(h, r):
    """Each query has one element of 1 to 2 and others of 2^-9 to 2^-14 of that, which decide the logits: the keys are 2^10
    times the usual and zero where the large element is."""
    sh = h["Q"].shape
    small = h["Q"] * 2.0 ** r.integers(-14, -8, sh)
    small[..., 0] = r.choice([-1.0, 1.0], sh[:-1]) * r.integers(128, 256, sh[:-1]) / 128.0
    h["Q"] = small
    h["K8"][..., 0] = 0
    h["ks"] = (h["ks"] * np.float32(2.0 ** 10)).astype(np.float32)


WIDE = (1, 8, 2, 100, 700, 128, 64, 5, 560, "bf16", "bf16", 710, wide_rows)
# The union kernel's loss on a small element is spread over +-2^-17 (root mean square 2^-17 / sqrt 3); a logit adds 127 of
# them times keys of 2^10 over sqrt 128: 2^-7 / sqrt 3.  A weight moves by that, an output (a sum of values of any sign) by as
# much of its root mean square; twice it is allowed, and 2^-8 for the result's and the weights' own rounding.
WIDE_TOL = {"union": 2 * 2.0 ** -7 / math.sqrt(3) + 2.0 ** -8, "rows": 2.0 ** -8}


def test_a_dropped_query_piece_is_seen():
    p, h = host_case(*WIDE)
    rows = range(0, 100, 5)
    want = compute(p, h, rows)
    assert rms_error(compute(p, h, rows, lambda q: query(q, "union")), want) <= WIDE_TOL["union"]
    assert rms_error(compute(p, h, rows, lambda q: query(q, "union", 1)), want) > WIDE_TOL["union"]
    assert rms_error(compute(p, h, rows, lambda q: query(q, "rows", 1)), want) <= WIDE_TOL["rows"]
    assert rms_error(compute(p, h, rows, lambda q: query(q, "union")), want) > WIDE_TOL["rows"] / 2


@pytest.mark.gpu
@pytest.mark.parametrize("kernel", ["rows", "union"])
def test_queries_with_one_large_element(kernel, monkeypatch):
    monkeypatch.setenv("HILS_Q8_KERNEL", kernel)
    p, h = host_case(*WIDE)
    O = c8.attend(p, on_device(p, h)).double().cpu().numpy()
    c8.ok()
    err = rms_error(O, compute(p, h))
    print("root mean square of the error %.3g, allowed %.3g" % (err, WIDE_TOL[kernel]))
    assert err <= WIDE_TOL[kernel]


# Float32 results.  Per output the roundings that are left: the query's and the weights' second pieces (2^-22 each at most),
# an exponential (2^-22), and about 42 float32 operations of 2^-24 on the way (a logit's eight partial sums, its factors, the
# sums over a chunk's keys and over the slots' blocks of 16 keys).  As squares: 2^-22 sqrt(3 + 42 / 16) < 2^-20.
F32_TOL = 2.0 ** -20


def truncated(a, b):
    """Float32 sums cut off instead of rounded, as an accumulator that a chain of products adds to would be."""
    s = a + b
    f = s.astype(np.float32).astype(np.float64)
    return np.where(np.abs(f) > np.abs(s), np.nextafter(f.astype(np.float32), np.float32(0.0)).astype(np.float64), f)


LONG = (1, 2, 1, 2, 128 * 68, 128, 128, 64, 128 * 67 + 60, "f32", "f32", 720)     # 65 chunks of 128 keys: 516 products a chain


def test_eleven_bits_and_truncated_chains_are_seen():
    p, h = host_case(1, 4, 2, 12, 1200, 64, 32, 8, 900, "f32", "f32", 721)
    want = compute(p, h)
    two = dict(q_as=lambda q: query(q, "rows"), p_as=lambda x: pieces(x, f16, 2))
    assert rms_error(compute(p, h, **two), want) <= F32_TOL / 2
    assert rms_error(compute(p, h, **dict(two, q_as=lambda q: query(q, "rows", 1))), want) > 8 * F32_TOL
    assert rms_error(compute(p, h, **dict(two, p_as=lambda x: pieces(x, f16, 1))), want) > 8 * F32_TOL
    p, h = host_case(*LONG)
    want = compute(p, h)
    assert rms_error(compute(p, h, **two), want) <= F32_TOL / 2
    assert rms_error(compute(p, h, **two, add=truncated), want) > 2 * F32_TOL


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("shape,share", [
    ((1, 4, 2, 12, 1200, 64, 32, 8, 900), 0), ((1, 4, 2, 12, 1200, 64, 64, 8, 900), 1), ((2, 12, 2, 6, 3000, 64, 128, 9, 2500), 8),
    ((1, 4, 2, 12, 1200, 128, 32, 8, 900), 1), ((1, 4, 2, 12, 1200, 128, 64, 8, 900), 8), ((2, 12, 2, 6, 3000, 128, 128, 9, 2500), 0),
    (LONG[:9], 0), (LONG[:9], 8)], ids=lambda s: "x".join(map(str, s)) if isinstance(s, tuple) else str(s))
def test_float32_results(shape, share, dtype, monkeypatch):
    """Every (d, C), lone warps, blocks and clusters; the longest chains of products there are."""
    monkeypatch.setenv("HILS_Q8_SHARE", str(share))
    p, h = host_case(*shape, dtype, "f32", 722)
    O = c8.attend(p, on_device(p, h)).double().cpu().numpy()
    c8.ok()
    err = rms_error(O, compute(p, h))
    print("root mean square of the error %.3g, allowed %.3g" % (err, F32_TOL))
    assert err <= F32_TOL


@pytest.mark.gpu
@pytest.mark.parametrize("d,C", [(64, 32), (64, 64), (64, 128), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("umul", [1.0, 8.0])
def test_float32_landmarks(d, C, umul):
    """The same measure: a chunk's probabilities over its keys, whose logits have a spread of umul.  A logit's error, 2^-22 of
    it, moves a weight by as much: umul of that."""
    r = np.random.default_rng(730 + d + C)
    B, Hkv, T = 2, 3, 11 * C + 7
    data, scale = c8.make_cache(r, B, Hkv, T, d, C, T, spread=2.0)
    nL = -(-T // C)
    U64, U = c8.rng_rows(r, (B, Hkv, nL, d), "f32", umul)
    # keys of 2^-2 to 2^2 times the usual: the landmark query goes with them (powers of two)
    level = scale / np.max(scale)
    U64, U = U64 / level[..., None], U / torch.from_numpy(level).to(c8.DEV)[..., None]
    p = hils.problem(B, Hkv, Hkv, 1, T, d, C, 0, 0, hils.HILS_F32)
    L, beta = torch.empty((B, Hkv, nL, d), device=c8.DEV), torch.empty((B, Hkv, nL), device=c8.DEV)
    hils.hils_landmarks_q8(p, torch.from_numpy(data).to(c8.DEV), torch.from_numpy(scale).to(c8.DEV), U, L, beta)
    c8.ok()
    want, wb = np.zeros((B, Hkv, nL, d)), np.zeros((B, Hkv, nL))
    for b in range(B):
        for g in range(Hkv):
            for c in range(nL):
                k = ref.TABLE[data[b, g, c * C:min((c + 1) * C, T)]] * float(scale[b, g, c])
                want[b, g, c], wb[b, g, c] = ref.landmarks(k, U64[b, g, c], 1.0 / math.sqrt(d))
    got = L.double().cpu().numpy() / level[..., None]
    err = rms_error(got, want / level[..., None])
    eb = math.sqrt(np.mean((beta.double().cpu().numpy() - wb) ** 2))
    print("landmarks %.3g of %.3g, entropies %.3g" % (err, F32_TOL * max(1.0, umul), eb))
    assert err <= F32_TOL * max(1.0, umul)
    assert eb <= F32_TOL * max(1.0, umul) * math.log(C)
