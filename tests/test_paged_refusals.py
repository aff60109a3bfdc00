"""Calls of the rotation and the append whose outputs are another tensor's
input or output too: refused before anything is launched, with no GPU."""
import ctypes

import pytest

from attention_forward_jvp_gb300 import binding, build

INVALID = 1
AT = [0x10000 * (i + 1) for i in range(8)]  # 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def L():
    build.build()
    return binding.lib()


@pytest.mark.parametrize("places", [
    [(0, 0), (0, 0)],          # one tensor in place, twice
    [(0, 2), (1, 2)],          # two into one
    [(0, 1), (1, 0)],          # exchanged
    [(0, 2), (1, 3), (4, 0)],  # the third into the first's input
    [(0, 1), (1, 2)],          # the first into the second's input
])
def test_rope_refuses_outputs_of_two(L, places):
    s = binding.AttnRopeSpec(AT[7], 64, 0, 1.0)
    t = (binding.AttnRopeTensor * len(places))()
    for a, (x, y) in zip(t, places):
        a.x, a.y, a.H = AT[x], AT[y], 2
        a.x_stride[:] = a.y_stride[:] = (512, 256, 64)
    for fn in (L.attn_rope, L.attn_rope_f16):
        assert fn(1, 4, 64, ctypes.byref(s), t, len(places), None, None, None, 0, 0, None) == INVALID


def _append(L, pools=(0, 1), k=2, v=3, q=4, q_out=5):
    c = binding.AttnPagedCache()
    c.B, c.max_pages, c.n_pages, c.page_size, c.Hkv, c.Dqk, c.Dv = 2, 4, 8, 16, 2, 64, 64
    c.k, c.v, c.page_table, c.seq_lens = AT[pools[0]], AT[pools[1]], AT[6], AT[7]
    c.k_stride[:], c.v_stride[:], c.table_stride = (2048, 1024, 64), (2048, 1024, 64), 4
    n = binding.AttnPagedNew()
    n.T, n.k, n.v, n.q, n.q_out, n.Hq = 2, AT[k], AT[v], AT[q], AT[q_out], 2
    for s in (n.k_stride, n.v_stride, n.q_stride, n.q_out_stride):
        s[:] = (128, 64)
    return [fn(ctypes.byref(c), ctypes.byref(n), None, None) for fn in (L.attn_paged_append, L.attn_paged_append_f16)]


@pytest.mark.parametrize("bad", [dict(pools=(0, 0)), dict(q_out=2), dict(q_out=3), dict(q=2, q_out=2)])
def test_append_refuses_outputs_of_two(L, bad):
    assert _append(L, **bad) == [INVALID, INVALID]
