"""Rotary positions and the paged cache without a GPU: the frequencies and
steps of the host functions, the oracle's pins, and what is refused before
anything is launched."""
import ctypes
import math
import os
import subprocess
from fractions import Fraction

import numpy as np
import pytest
import torch

from attention_forward_jvp_gb300 import binding, build
from oracle import paged_ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID, UNSUPPORTED, MISALIGNED = 1, 2, 3
FAKE = 0x10000  # 16-byte aligned, never dereferenced: every call here is refused or empty


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


# ------------------------------------------------------------------- oracle
def test_oracle_rope_by_hand():
    # pair (3, 4) by a right angle: (-4, 3); the third element is not turned
    x = np.array([[3.0, 4.0, 7.0]])
    np.testing.assert_allclose(paged_ref.rope(x, [2], [math.pi / 4], interleaved=True), [[-4.0, 3.0, 7.0]], atol=1e-15)
    x = np.array([[1.0, 10.0, 2.0, 20.0]])  # pairs (1, 2) and (10, 20), the second at rest
    np.testing.assert_allclose(paged_ref.rope(x, [1], [math.pi / 2, 0.0], out_scale=0.5), [[-1.0, 5.0, 0.5, 10.0]],
                               atol=1e-15)


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rope_gradient_by_differences(interleaved):
    r = np.random.RandomState(0)
    w = paged_ref.rope_frequencies(6)
    x, g, d = r.randn(3, 5, 8), r.randn(3, 5, 8), r.randn(3, 5, 8)
    pos = [0, 1, 7, 1000, 131071]
    f = lambda z: float((paged_ref.rope(z, pos, w, interleaved, 1.3) * g).sum())  # noqa: E731
    grad = paged_ref.rope(g, pos, w, interleaved, 1.3, inverse=True)
    eps = 1e-3  # linear: only rounding is left
    assert abs((f(x + eps * d) - f(x - eps * d)) / (2 * eps) - float((grad * d).sum())) < 1e-9


def test_oracle_rope_scores_depend_on_distance_alone():
    r = np.random.RandomState(1)
    q, k = r.randn(1, 16), r.randn(1, 16)
    w = paged_ref.rope_frequencies(16)
    at = lambda p, j: float((paged_ref.rope(q, [p], w) * paged_ref.rope(k, [j], w)).sum())  # noqa: E731
    assert abs(at(5, 2) - at(1005, 1002)) < 1e-11


def test_oracle_decode_by_hand():
    # one key: its value, lse = s q k; two equal keys: the mean, lse + log 2
    kp = np.zeros((3, 1, 2, 2))
    vp = np.zeros((3, 1, 2, 2))
    kp[2, 0, 0], vp[2, 0, 0] = [1.0, 2.0], [5.0, 7.0]
    kp[2, 0, 1], vp[2, 0, 1] = [1.0, 2.0], [1.0, 1.0]
    q = np.array([[[3.0, 4.0]]])
    o, lse = paged_ref.decode(q, kp, vp, np.array([[2]]), [1], sm_scale=0.5)
    np.testing.assert_allclose(o, [[[5.0, 7.0]]])
    np.testing.assert_allclose(lse, [[5.5]])
    o, lse = paged_ref.decode(q, kp, vp, np.array([[2]]), [2], sm_scale=0.5)
    np.testing.assert_allclose(o, [[[3.0, 4.0]]])
    np.testing.assert_allclose(lse, [[5.5 + math.log(2)]])
    o, lse = paged_ref.decode(q, kp, vp, np.array([[2]]), [0])
    assert (o == 0).all() and np.isneginf(lse).all()


# -------------------------------------------------------------- frequencies
def _freqs(L, rot, base=10000.0, scaling=0, factor=1.0, orig=0.0, low=1.0, high=32.0):
    f = binding.AttnRopeFreq(rot, scaling, base, factor, orig, low, high)
    out = np.full(max(rot, 2) // 2, np.nan)
    return L.attn_rope_freqs(ctypes.byref(f), out.ctypes.data), out


@pytest.mark.parametrize("rot", [2, 6, 64, 128])
@pytest.mark.parametrize("scaling", [None, "linear", "base", "by_parts"])
def test_frequencies(L, rot, scaling):
    if rot == 2 and scaling == "base":
        assert _freqs(L, rot, scaling=2, factor=4.0)[0] == INVALID
        return
    kw = dict(base=500000.0, scaling=scaling, factor=8.0, orig_len=8192, low_turns=1.0, high_turns=4.0)
    st, got = _freqs(L, rot, 500000.0, binding._ROPE_SCALING[scaling], 8.0, 8192, 1.0, 4.0)
    assert st == 0
    np.testing.assert_allclose(got, paged_ref.rope_frequencies(rot, **kw), rtol=1e-13)


def test_frequency_refusals(L):
    assert L.attn_rope_freqs(None, None) == INVALID
    for bad in (dict(rot=0), dict(rot=7), dict(rot=8, base=0.0), dict(rot=8, base=math.inf), dict(rot=8, scaling=4),
                dict(rot=8, scaling=-1), dict(rot=8, scaling=1, factor=0.0), dict(rot=8, scaling=3, factor=2.0),
                dict(rot=8, scaling=3, factor=2.0, orig=4096.0, low=4.0, high=4.0),
                dict(rot=8, scaling=2, base=1e300, factor=1e300), dict(rot=8, scaling=1, factor=5e-324)):
        assert _freqs(L, **bad)[0] == INVALID, bad


@pytest.mark.parametrize("w", [0.0, 1.0, 1e-6, math.pi, 2 * math.pi, 7.5, -1.0, -1e-9, 0.1 ** 7])
def test_steps_are_turns(L, w):
    f, s = np.array([w]), np.zeros(1, dtype=np.uint64)
    assert L.attn_rope_steps(f.ctypes.data, 1, s.ctypes.data) == 0
    # position 2^20: the fraction of a turn, in rational arithmetic; the turn
    # w / 2 pi is held to 2^-53 relative (absolute once it has wrapped)
    p = 1 << 20
    got = ((p * int(s[0])) % (1 << 64)) / 2.0**64
    turn = Fraction(w) * p / Fraction(2 * math.pi)
    want = float(turn - math.floor(turn))
    tol = p * 2.0**-52 * max(abs(w) / 6.28, 1.0 if w < 0 else 2.0**-11)
    assert min(abs(got - want), 1 - abs(got - want)) <= tol


def test_steps_refusals(L):
    s = np.zeros(1, dtype=np.uint64)
    for bad in (math.nan, math.inf):
        f = np.array([bad])
        assert L.attn_rope_steps(f.ctypes.data, 1, s.ctypes.data) == INVALID
    assert L.attn_rope_steps(None, 1, s.ctypes.data) == INVALID
    assert L.attn_rope_steps(None, 0, None) == 0


# ----------------------------------------------------------------- refusals
def _rope_call(L, B=1, N=4, D=64, rot=64, n=1, steps=FAKE, scale=1.0, x=FAKE, y=FAKE + 4096, H=2, xs=(512, 256, 64),
               ys=(512, 256, 64), offsets=None, n_seq=0, positions=None, ps=None, spec=True):
    s = binding.AttnRopeSpec(steps, rot, 0, scale)
    t = (binding.AttnRopeTensor * 4)()
    for a in t:
        a.x, a.y, a.H = x, y, H
        a.x_stride[:], a.y_stride[:] = xs, ys
    return L.attn_rope(B, N, D, ctypes.byref(s) if spec else None, t, n, positions, ps, offsets, n_seq, 0, None)


@pytest.mark.parametrize("bad,want", [
    (dict(spec=False), INVALID), (dict(B=-1), INVALID), (dict(N=-1), INVALID), (dict(n=0), INVALID),
    (dict(n=5), INVALID), (dict(D=0), UNSUPPORTED), (dict(D=1025), UNSUPPORTED), (dict(rot=66), INVALID),
    (dict(rot=7), INVALID), (dict(rot=0), INVALID), (dict(steps=None), INVALID), (dict(steps=FAKE + 4), MISALIGNED),
    (dict(scale=math.inf), INVALID), (dict(scale=math.nan), INVALID), (dict(x=None), INVALID), (dict(y=None), INVALID),
    (dict(x=FAKE + 1), MISALIGNED), (dict(H=-1), INVALID), (dict(y=FAKE, ys=(512, 64, 128)), INVALID),
    (dict(B=2, offsets=FAKE, n_seq=1), INVALID), (dict(offsets=FAKE, n_seq=-1), INVALID),
    (dict(offsets=FAKE + 2, n_seq=1), MISALIGNED), (dict(positions=FAKE), INVALID), (dict(N=1 << 31), INVALID),
    (dict(ys=(512, 0, 64)), INVALID), (dict(ys=(512, 256, 0)), INVALID),
    (dict(y=FAKE, xs=(512, 0, 64), ys=(512, 0, 64)), INVALID)])
def test_rope_refuses(L, bad, want):
    assert _rope_call(L, **bad) == want


def test_rope_of_nothing(L):
    assert _rope_call(L, B=0, x=None) == 0
    assert _rope_call(L, N=0, x=None) == 0
    assert _rope_call(L, H=0, x=None) == 0
    assert _rope_call(L, offsets=FAKE, n_seq=0, x=None) == 0


def _cache(**kw):
    c = binding.AttnPagedCache()
    c.B, c.max_pages, c.n_pages, c.page_size, c.Hkv, c.Dqk, c.Dv = 2, 4, 8, 16, 2, 64, 64
    c.k = c.v = c.page_table = c.seq_lens = FAKE
    c.k_stride[:], c.v_stride[:], c.table_stride = (2048, 1024, 64), (2048, 1024, 64), 4
    for k, v in kw.items():
        if k in ("k_stride", "v_stride"):
            getattr(c, k)[:] = v
        else:
            setattr(c, k, v)
    return c


CACHE_REFUSALS = [
    (dict(B=-1), INVALID), (dict(max_pages=-1), INVALID), (dict(n_pages=-1), INVALID), (dict(page_size=0), INVALID),
    (dict(Hkv=0), INVALID), (dict(Dqk=48), UNSUPPORTED), (dict(Dv=512), UNSUPPORTED), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(seq_lens=None), INVALID), (dict(page_table=None), INVALID),
    (dict(k=FAKE + 8), MISALIGNED), (dict(v=FAKE + 2), MISALIGNED), (dict(k_stride=(2048, 1024, 68)), MISALIGNED),
    (dict(v_stride=(2044, 1024, 64)), MISALIGNED), (dict(seq_lens=FAKE + 2), MISALIGNED)]


def _decode_call(L, c, Hq=4, q=FAKE, qs=(256, 64), scale=math.nan, o=FAKE, lse=FAKE, ws=FAKE, n=1 << 40):
    return L.attn_paged_decode(ctypes.byref(c) if c is not None else None, Hq, q,
                               (ctypes.c_int64 * 2)(*qs) if qs else None, scale, o, lse, ws, n, None)


def _append_call(L, c, rope=None, **kw):
    n = binding.AttnPagedNew()
    n.T, n.k, n.v, n.q, n.q_out, n.Hq = 2, FAKE, FAKE, FAKE, FAKE, 4
    n.k_stride[:], n.v_stride[:], n.q_stride[:], n.q_out_stride[:] = (128, 64), (128, 64), (256, 64), (256, 64)
    for k, v in kw.items():
        if k.endswith("_stride"):
            getattr(n, k)[:] = v
        else:
            setattr(n, k, v)
    return L.attn_paged_append(ctypes.byref(c) if c is not None else None, ctypes.byref(n), rope, None)


@pytest.mark.parametrize("bad,want", CACHE_REFUSALS)
def test_cache_refused(L, bad, want):
    c = _cache(**bad)
    assert _decode_call(L, c) == want
    assert _append_call(L, c) == want
    assert L.attn_paged_decode_workspace(ctypes.byref(c), 4) == 0


@pytest.mark.parametrize("bad,want", [
    (dict(Hq=-1), INVALID), (dict(Hq=3), INVALID), (dict(q=None), INVALID), (dict(qs=None), INVALID),
    (dict(o=None), INVALID), (dict(lse=None), INVALID), (dict(ws=None), INVALID), (dict(scale=0.0), INVALID),
    (dict(scale=-1.0), INVALID), (dict(scale=math.inf), INVALID), (dict(q=FAKE + 8), MISALIGNED),
    (dict(qs=(256, 60)), MISALIGNED), (dict(o=FAKE + 8), MISALIGNED), (dict(lse=FAKE + 2), MISALIGNED),
    (dict(ws=FAKE + 8), MISALIGNED)])
def test_decode_refuses(L, bad, want):
    assert _decode_call(L, None) == INVALID
    assert _decode_call(L, _cache(), **bad) == want


@pytest.mark.parametrize("bad,want", [
    (dict(T=-1), INVALID), (dict(T=3), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID),
    (dict(q_out=None), INVALID), (dict(Hq=-1), INVALID), (dict(k=FAKE + 1), MISALIGNED),
    (dict(offsets=FAKE + 2), MISALIGNED), (dict(q_out_stride=(512, 64)), INVALID),
    (dict(q_stride=(256, 0), q_out_stride=(256, 0)), INVALID)])
def test_append_refuses(L, bad, want):
    assert _append_call(L, None) == INVALID
    assert _append_call(L, _cache(), **bad) == want


@pytest.mark.parametrize("strides", [(0, 1024, 64), (2048, 0, 64), (2048, 1024, 0)])
def test_append_refuses_pools_that_share_places(L, strides):
    assert _append_call(L, _cache(k_stride=strides)) == INVALID
    assert _append_call(L, _cache(v_stride=strides)) == INVALID


def test_append_refuses_a_wide_rotation(L):
    s = binding.AttnRopeSpec(FAKE, 66, 0, 1.0)
    assert _append_call(L, _cache(), ctypes.byref(s)) == INVALID


def test_empty_calls_touch_nothing(L):
    assert _decode_call(L, _cache(B=0, seq_lens=None), q=None, o=None) == 0
    assert _decode_call(L, _cache(), Hq=0, q=None, o=None) == 0
    assert _append_call(L, _cache(B=0, seq_lens=None), T=0, k=None) == 0
    assert _append_call(L, _cache(), T=0, offsets=FAKE, k=None) == 0


def test_binding_refuses_cpu_tensors_and_bad_rotations():
    z = torch.zeros(1, 1, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.PagedCache(z, z, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        binding.PagedCache(*(torch.zeros(1) for _ in range(4)))
    for bad in (dict(rot_dim=7), dict(rot_dim=8, scaling="cubic"), dict(rot_dim=8, out_scale=math.inf),
                dict(rot_dim=8, inv_freq=[1.0, 2.0]), dict(rot_dim=4, inv_freq=[1.0, 2.0], scaling="linear"),
                dict(rot_dim=8, device="cpu")):
        with pytest.raises(ValueError):
            binding.Rope(**bad)
    with pytest.raises(binding.AttnError):
        binding.Rope(8, scaling="linear", factor=-1.0)


def test_abi_from_c(tmp_path):
    """A C99 caller through attn_paged.h; it prints its failed checks."""
    build.build()
    exe = tmp_path / "paged_from_c"
    libdir = os.path.dirname(build.LIB_PATH)
    subprocess.run(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.join(ROOT, "include"),
                    os.path.join(ROOT, "tests", "c", "paged_from_c.c"), "-o", str(exe), "-L", libdir, "-lattn_jvp",
                    f"-Wl,-rpath,{libdir}", "-lm"], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout + r.stderr
