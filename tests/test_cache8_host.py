"""The 8-bit cache's entry points refuse what they do not cover before any launch (CPU), and the reference encoder that
the GPU tests compare with is itself pinned."""
import numpy as np
import pytest

import cache8_ref as ref
import chunk_wise_hierarchical_hils_b200 as hils

OK, INV, UNS, WS = hils.HILS_OK, hils.HILS_ERR_INVALID_ARG, hils.HILS_ERR_UNSUPPORTED, hils.HILS_ERR_WORKSPACE


def prob(**kw):
    base = dict(B=2, H=8, Hkv=2, N=256, T=256, d=128, C=64, k=4)
    base.update(kw)
    return hils.problem(**base)


def status(fn, *a, **kw):
    try:
        fn(*a, **kw)
    except hils.HilsError as e:
        return e.status
    return OK


@pytest.mark.parametrize("call", ["append", "read"])
@pytest.mark.parametrize("kw,ptrs,rng,want", [
    ({}, {}, (5, 5), OK),                                  # an empty range launches nothing
    ({"H": 3, "N": 0, "k": -1}, {}, (0, 0), OK),           # fields the calls do not use may hold anything
    ({}, {}, (256, 256), OK),
    ({}, {}, (-1, 4), INV),
    ({}, {}, (6, 5), INV),
    ({}, {}, (0, 257), INV),                               # past the capacity
    ({"B": 0}, {}, (0, 1), INV),
    ({"T": 0}, {}, (0, 0), INV),
    ({"C": 0}, {}, (0, 1), INV),
    ({"C": 48}, {}, (0, 1), UNS),
    ({"d": 96}, {}, (0, 1), UNS),
    ({"in_dtype": 5}, {}, (0, 1), INV),
    ({"B": 65536, "Hkv": 1, "H": 1}, {}, (0, 1), UNS),
    ({}, {0: None}, (0, 1), INV), ({}, {1: None}, (0, 1), INV), ({}, {2: None}, (0, 1), INV),
    ({}, {3: None}, (0, 1), INV), ({}, {4: None}, (0, 1), INV), ({}, {5: None}, (0, 1), INV),
    ({}, {0: 24}, (0, 1), INV), ({}, {1: 24}, (0, 1), INV), ({}, {2: 24}, (0, 1), INV), ({}, {3: 24}, (0, 1), INV),
    ({}, {4: 18}, (0, 1), INV), ({}, {5: 18}, (0, 1), INV),
])
def test_append_and_read_refusals(call, kw, ptrs, rng, want):
    fn = hils.hils_cache_append_q8 if call == "append" else hils.hils_cache_read_q8
    a = [16, 32, 48, 64, 80, 96] if call == "append" else [16, 32, 80, 96, 48, 64]
    for i, v in ptrs.items():
        # positions are given for append: K, V, K8, V8, k_scale, v_scale; read takes K8, V8, k_scale, v_scale, K, V
        a[i if call == "append" else (4, 5, 0, 1, 2, 3)[i]] = v
    assert status(fn, prob(**kw), *a, *rng, stream=0) == want


@pytest.mark.parametrize("kw,a,want", [
    ({}, (16, 16, 16, 32, None, 2, 2, 256), OK),
    ({}, (16, 16, 16, 32, None, 1, 1, 65), OK),
    ({}, (16, 16, 16, 32, None, 0, 2, 64), INV),           # chunk 1 holds no token yet
    ({}, (16, 16, 16, 32, None, 0, 1, 0), INV),
    ({}, (16, 16, 16, 32, None, 0, 1, 257), INV),
    ({}, (16, 16, 16, 32, None, -1, 1, 64), INV),
    ({}, (16, 16, 16, 32, None, 2, 1, 256), INV),
    ({"C": 7}, (16, 16, 16, 32, None, 0, 1, 64), UNS),
    ({"d": 32}, (16, 16, 16, 32, None, 0, 1, 64), UNS),
    ({"scale": float("inf")}, (16, 16, 16, 32, None, 0, 1, 64), INV),
    ({}, (None, 16, 16, 32, None, 0, 1, 64), INV),
    ({}, (16, None, 16, 32, None, 0, 1, 64), INV),
    ({}, (16, 16, None, 32, None, 0, 1, 64), INV),
    ({}, (16, 16, 16, None, None, 0, 1, 64), INV),
    ({}, (24, 16, 16, 32, None, 0, 1, 64), INV),
    ({}, (16, 18, 16, 32, None, 0, 1, 64), INV),
    ({}, (16, 16, 24, 32, None, 0, 1, 64), INV),
    ({}, (16, 16, 16, 24, None, 0, 1, 64), INV),
    ({}, (16, 16, 16, 32, 18, 0, 1, 64), INV),
])
def test_landmarks_refusals(kw, a, want):
    assert status(hils.hils_landmarks_q8, prob(**kw), *a, stream=0) == want


BASE = [16, 32, 48, 64, 80, 96, 112, 128]                  # Q, K8, V8, k_scale, v_scale, sel_idx, sel_score, O


@pytest.mark.parametrize("kw,ptrs,want", [
    ({"d": 96}, {}, UNS), ({"C": 16}, {}, UNS), ({"k": 65}, {}, UNS), ({"H": 34}, {}, UNS), ({"H": 7}, {}, INV),
    ({"N": 0}, {}, INV), ({"q_offset": 1}, {}, INV), ({"scale": -1.0}, {}, INV), ({"out_dtype": 9}, {}, INV),
    *[({}, {i: None}, INV) for i in range(8)],
    *[({}, {i: 24}, INV) for i in (0, 1, 2, 5, 6, 7)],
    *[({}, {i: 18}, INV) for i in (3, 4)],
])
def test_attend_refusals(kw, ptrs, want):
    a = list(BASE)
    for i, v in ptrs.items():
        a[i] = v
    assert status(hils.hils_chunk_attend_fuse_q8, prob(**kw), *a, (16, 1 << 40), stream=0) == want


def test_forward_refusals():
    p = prob()
    need = hils.hils_forward_q8_workspace_size(p)
    assert need >= 2 * 2 * 256 * 4 * 4 + 2 * 8 * 256 * 5 * 4
    args = [16, 32, 48, 64, 80, 96, 112]                   # Q, K8, V8, k_scale, v_scale, L, O
    assert status(hils.hils_forward_q8, p, *args, (16, need - 1), stream=0) == WS
    assert status(hils.hils_forward_q8, p, *args, (24, need), stream=0) == INV
    assert status(hils.hils_forward_q8, p, *args, None, stream=0) == WS
    for i in range(7):
        assert status(hils.hils_forward_q8, p, *args[:i], None, *args[i + 1:], (16, need), stream=0) == INV
        assert status(hils.hils_forward_q8, p, *args[:i], args[i] + 2, *args[i + 1:], (16, need), stream=0) == INV
    with pytest.raises(hils.HilsError):
        hils.hils_forward_q8_workspace_size(prob(d=80))
    with pytest.raises(hils.HilsError):
        hils.hils_chunk_attend_fuse_q8_workspace_size(prob(C=20))


def test_attend_short_workspace():
    for kw in (dict(), dict(N=1, T=4096, q_offset=4095, k=32), dict(B=1, H=32, Hkv=8, N=4096, T=4096, k=16)):
        p = prob(**kw)
        need = hils.hils_chunk_attend_fuse_q8_workspace_size(p)
        if need:
            assert status(hils.hils_chunk_attend_fuse_q8, p, *BASE, (16, need - 1), stream=0) == WS
            assert status(hils.hils_chunk_attend_fuse_q8, p, *BASE, None, stream=0) == WS
            assert status(hils.hils_chunk_attend_fuse_q8, p, *BASE, (8, need), stream=0) == INV


def test_reference_encoder():
    # every byte is its own nearest value, midpoints go to the even code, the range saturates
    b = np.arange(256)
    keep = (b & 127) != 127
    assert np.array_equal(ref.encode(ref.TABLE[b])[keep], b[keep])
    assert np.all(ref.encode(ref.TABLE[b])[~keep] == 127)
    pos = ref.TABLE[:127]
    assert np.all(np.diff(pos) > 0) and pos[1] == 2.0 ** -9 and pos[126] == 448.0
    mid = (pos[:-1] + pos[1:]) / 2
    code = ref.encode(mid)
    assert np.all(code % 2 == 0) and np.all(np.abs(code.astype(int) - np.arange(126)) <= 1)
    assert np.array_equal(ref.encode(np.nextafter(mid, 0)), np.arange(126))
    assert np.array_equal(ref.encode(np.nextafter(mid, 1e9)), np.arange(1, 127))
    assert list(ref.encode(np.array([1e9, -np.inf, np.nan, -0.0]))) == [126, 254, 127, 128]


def test_reference_scale():
    assert ref.scale_for(0.0) == 2.0 ** -100 and ref.scale_for(448.0) == 1.0 and ref.scale_for(448.0001) == 2.0
    assert ref.scale_for(3.4e38) == 2.0 ** 119
