"""Rotary positions, paged append and paged decode on the GPU against the
float64 definitions of oracle.paged_ref.

Tolerances, from the arithmetic (u = half a step of the output type,
torch.finfo(t).eps / 2):

  rope    u |y| for the output's rounding, and 1e-6 out_scale (|a| + |b|):
          the angle's fraction of half a turn is rounded to fp32
          (pi 2^-25 = 9.4e-8), sincospif is good to 2 ulp (2.4e-7), products
          and sum round three times (1.8e-7).  A subnormal step for fp16.
  decode  scores: d = (Dqk + 4) 2^-22 s max_j sum |q| |k_j| (fp32 sums, a
          rounding and a truncation each); a weight is off by 2 d (its own
          score's error and the others') + 2^-15 (exp2, and the two 16-bit
          parts of P), so O by (2 d + 2^-15) sum_j w_j |V_j|, and u |O|; fp16
          weights below 2^-14 lose up to 2^-25 each, n 2^-25 max|V| in all.
          LSE: d + (n + 8) 2^-24 + 2^-21 |LSE|.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from attention_forward_jvp_gb300 import binding, build
from oracle import paged_ref

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    binding.lib()


@pytest.fixture(autouse=True)
def _clean(_lib):
    assert binding.sync_check() == 0
    yield


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(shape, dtype, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).to(dtype).cuda()


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.int16), b.contiguous().view(torch.int16))


# --------------------------------------------------------------------- rope
def check_rope(y, x, pos, r, inverse=False, what=""):
    """y, x [..., N, D] tensors, pos N positions."""
    X = f64(x)
    want = paged_ref.rope(X, pos, f64(r.inv_freq), r.interleaved, r.out_scale, inverse)
    half = r.rot_dim // 2
    size = np.zeros_like(X)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if r.interleaved else (i, i + half)
    size[..., a] = size[..., b] = np.abs(X[..., a]) + np.abs(X[..., b])
    tol = torch.finfo(y.dtype).eps / 2 * np.abs(want) + 1e-6 * abs(r.out_scale) * size
    tol += 2.0**-25 if y.dtype == HF else 2.0**-130
    tol[..., r.rot_dim:] = 0  # copied
    err = np.abs(f64(y) - want)
    assert not np.isnan(err).any(), what
    assert (err <= tol).all(), f"{what}: worst {np.max(err - tol):.3e} over its bound"


ROPES = [  # D, rot_dim, interleaved, dtype
    (128, 128, False, BF), (128, 128, True, BF), (64, 32, False, HF), (64, 32, True, HF), (256, 64, False, BF),
    (16, 16, True, BF), (32, 8, False, BF), (80, 20, True, HF), (64, 2, False, BF), (1024, 1024, False, HF),
    (7, 6, True, BF), (96, 48, False, BF)]


@pytest.mark.parametrize("D,rot,inter,dt", ROPES)
@pytest.mark.parametrize("inverse", [False, True])
def test_rope_dense(D, rot, inter, dt, inverse):
    r = binding.Rope(rot, interleaved=inter, out_scale=1.25)
    x = [randn((2, h, 37, D), dt, 10 * D + i) for i, h in enumerate((3, 1, 6, 2))]
    y = binding.attn_rope(x, r, inverse=inverse)
    for a, b in zip(x, y):
        assert b.is_contiguous()
        check_rope(b, a, range(37), r, inverse)
    assert binding.sync_check() == 0


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("scaling", [None, "linear", "base", "by_parts"])
def test_rope_far_positions_and_scalings(inter, scaling):
    r = binding.Rope(64, base=500000.0, interleaved=inter, scaling=scaling, factor=8.0, orig_len=8192, low_turns=1.0,
                     high_turns=4.0)
    pos = [0, 1, 4095, 65537, 131071, 1048576, 2**24 + 1, -1, -70000]
    x = randn((1, 2, len(pos), 64), BF, 5)
    y, = binding.attn_rope([x], r, positions=torch.tensor(pos, dtype=torch.int32).cuda())
    check_rope(y, x, pos, r)


def test_rope_given_frequencies():
    r = binding.Rope(8, inv_freq=[0.0, 3.5, -0.25, 7.0])
    x = randn((1, 1, 40, 16), HF, 6)
    y, = binding.attn_rope([x], r)
    check_rope(y, x, range(40), r)


@pytest.mark.parametrize("N", [1, 2, 33, 1000])
def test_rope_views_positions_and_in_place(N):
    # q and k out of one packed [B, N, heads, D] projection, positions per batch entry
    r = binding.Rope(64, interleaved=False)
    packed = randn((3, N, 9, 64), BF, N)
    q, k = packed[:, :, :4].transpose(1, 2), packed[:, :, 4:6].transpose(1, 2)
    pos = torch.randint(0, 100000, (3, N), dtype=torch.int32).cuda()
    before = packed.clone()
    y = binding.attn_rope([q, k], r, positions=pos)
    assert torch.equal(packed, before)
    for b in range(3):
        check_rope(y[0][b], q[b], pos[b].tolist(), r)
        check_rope(y[1][b], k[b], pos[b].tolist(), r)
    z = binding.attn_rope([q, k], r, positions=pos, out=[q, k])
    assert torch.equal(z[0], y[0]) and torch.equal(z[1], y[1])
    assert torch.equal(packed[:, :, 6:], before[:, :, 6:])


@pytest.mark.parametrize("shift", [1, 4, 8])
def test_rope_unaligned_rows_equal_aligned_ones(shift):
    r = binding.Rope(32, interleaved=shift == 4)
    x = randn((2, 3, 21, 64), BF, shift)
    y, = binding.attn_rope([x], r)
    buf = torch.full((2, 3, 21, 64 + 9), float("nan"), dtype=BF, device="cuda")
    v = buf[..., shift:shift + 64]
    v.copy_(x)
    z, = binding.attn_rope([v], r, out=[v])
    assert torch.equal(z, y)
    assert buf[..., :shift].isnan().all() and buf[..., shift + 64:].isnan().all()


@pytest.mark.parametrize("lens,T", [([5, 0, 17, 1, 0], 30), ([0, 0], 4), ([64], 64), ([1] * 70, 70), ([300, 2, 900], 1202)])
@pytest.mark.parametrize("inter,given", [(False, False), (True, True)])
def test_rope_jagged(lens, T, inter, given):
    off = torch.tensor([0] + lens).cumsum(0).int().cuda()
    r = binding.Rope(64, interleaved=inter)
    x = [randn((h, T, 64), HF, 3 + h) for h in (4, 2)]
    out = [torch.full_like(t, float("nan")) for t in x]
    pos = [p for n in lens for p in range(n)]
    arg = None
    if given:
        pos = [7 * p + 3 for p in pos]
        arg = torch.tensor(pos + [0] * (T - len(pos)), dtype=torch.int32).cuda()
    y = binding.attn_rope(x, r, positions=arg, offsets=off, out=out)
    n = len(pos)
    for a, b in zip(x, y):
        if n:
            check_rope(b[:, :n], a[:, :n], pos, r)
        assert b[:, n:].isnan().all()


def test_rope_of_tensors_given_twice():
    r = binding.Rope(64)
    q, k = randn((2, 6, 9, 64), BF, 0), randn((2, 2, 9, 64), BF, 1)
    (a,), (b,) = binding.attn_rope([q], r), binding.attn_rope([k], r)
    for x, want in zip(binding.attn_rope([q, k, q, k], r), (a, b, a, b)):
        assert torch.equal(x, want)


def test_rope_inverse_transposes():
    # <R x, g> = <x, R^T g>: each side sums products whose rounded factor is
    # off by u relative (2^-11)
    r = binding.Rope(64, out_scale=0.75)
    x, g = randn((2, 4, 50, 64), HF, 1), randn((2, 4, 50, 64), HF, 2)
    y, = binding.attn_rope([x], r)
    gx, = binding.attn_rope([g], r, inverse=True)
    a, b = f64(y) * f64(g), f64(x) * f64(gx)
    assert abs(a.sum() - b.sum()) <= 2.0**-11 * (np.abs(a).sum() + np.abs(b).sum()) + 1e-6 * x.numel()


def test_rope_gradient_by_differences():
    # along a direction d, of L = sum(g o rope(x)): the map is linear, so
    # (L(x + d) - L(x - d)) / 2 = <R^T g, d> but for the roundings of the two
    # outputs (2^-11 |y| each) and of the gradient
    r = binding.Rope(32, interleaved=True)
    x, g, d = ((randn((1, 2, 30, 32), torch.float32, s) * 64).round().div(64).to(HF) for s in (1, 2, 3))
    assert torch.equal((x + d).double(), x.double() + d.double())  # no rounding in the arguments
    up, down = binding.attn_rope([x + d, x - d], r)
    gx, = binding.attn_rope([g], r, inverse=True)
    diff = ((f64(up) - f64(down)) / 2 * f64(g)).sum()
    want = (f64(gx) * f64(d)).sum()
    tol = 2.0**-11 * ((np.abs(f64(up)) + np.abs(f64(down))) / 2 * np.abs(f64(g))).sum()
    tol += 2.0**-11 * np.abs(f64(gx) * f64(d)).sum() + 4e-6 * x.numel()
    assert abs(diff - want) <= tol


def test_rope_nonfinite_values_stay_in_their_pairs():
    r = binding.Rope(32, interleaved=False)
    x = randn((1, 1, 4, 64), BF, 8)
    y0, = binding.attn_rope([x], r)
    x[0, 0, 2, 5] = float("inf")
    x[0, 0, 3, 40] = float("nan")
    y, = binding.attn_rope([x], r)
    bad = ~torch.isfinite(y[0, 0])
    assert set(map(tuple, bad.nonzero().tolist())) <= {(2, 5), (2, 21), (3, 40)} and bad[3, 40] and bad[2].any()
    assert torch.equal(y[0, 0][~bad], y0[0, 0][~bad])


def test_rope_refusals():
    r = binding.Rope(64)
    x = randn((1, 2, 4, 64), BF, 0)
    for bad in (lambda: binding.attn_rope([], r), lambda: binding.attn_rope([x] * 5, r),
                lambda: binding.attn_rope([x[0]], r), lambda: binding.attn_rope([x, x[:, :, :3]], r),
                lambda: binding.attn_rope([x.cpu()], r), lambda: binding.attn_rope([x, x.transpose(1, 2)], r),
                lambda: binding.attn_rope([randn((1, 2, 64, 64), BF, 0).transpose(2, 3)], r),
                lambda: binding.attn_rope([x], binding.Rope(128)), lambda: binding.attn_rope([x], r, out=[x[:, :1]]),
                lambda: binding.attn_rope([x], r, out=[]),
                lambda: binding.attn_rope([x], r, positions=torch.zeros(5, dtype=torch.int32, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: binding.attn_rope([x.float()], r), lambda: binding.attn_rope([x, x.half()], r),
                lambda: binding.attn_rope([x], r, positions=torch.zeros(4, dtype=torch.int64, device="cuda")),
                lambda: binding.attn_rope([x[0]], r, offsets=torch.zeros(2, dtype=torch.int64, device="cuda"))):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(binding.AttnError):  # in place by other strides
        binding.attn_rope([x], r, out=[x.view(1, 4, 2, 64).transpose(1, 2)])


# -------------------------------------------------------------------- cache
class Pool:
    """Pools of pages in a shuffled order; what is behind each sequence's
    last token, and in pages of nobody, is NaN; so are the table's entries
    behind a sequence's last page numbers of no use (out of range)."""

    def __init__(self, lens, Hkv, Dqk, Dv, page, dtype, seed=0, head_major=True, std=1.0, extra=2):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        count = sum(need) + 2
        order = torch.randperm(count, generator=g)
        self.lens, self.page = lens, page
        pools = [torch.full((count, Hkv, page, d), float("nan"), dtype=dtype) for d in (Dqk, Dv)]
        table = torch.full((len(lens), max(need + [1]) + extra), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n].int()
            for j in range(n):
                m = min(page, lens[b] - j * page)
                for p in pools:
                    p[order[at + j], :, :m] = (torch.randn((Hkv, m, p.shape[3]), generator=g) * std).to(dtype)
            at += n
        if not head_major:  # token-major storage, seen as [pages, heads, page, d]
            pools = [p.transpose(1, 2).contiguous() for p in pools]
        self.k, self.v = (p.cuda() if head_major else p.cuda().transpose(1, 2) for p in pools)
        self.table, self.seq_lens = table.cuda(), torch.tensor(lens, dtype=torch.int32).cuda()
        self.cache = binding.PagedCache(self.k, self.v, self.table, self.seq_lens)


def check_decode(pool, q, o, lse, sm_scale=None):
    K, V, table, Q = f64(pool.k), f64(pool.v), pool.table.cpu().numpy(), f64(q)
    want, wl = paged_ref.decode(Q, K, V, table, pool.lens, sm_scale)
    B, Hq, Dqk = Q.shape
    Hkv, page = K.shape[1], K.shape[2]
    s = Dqk**-0.5 if sm_scale is None else sm_scale
    O, L = f64(o), f64(lse)
    assert np.isfinite(O).all() and not np.isnan(L).any()
    u = torch.finfo(o.dtype).eps / 2
    for b in range(B):
        n = int(pool.lens[b])
        if n == 0:
            assert (O[b] == 0).all() and np.isneginf(L[b]).all()
            continue
        at = np.arange(n)
        pages, slots = table[b, at // page], at % page
        for h in range(Hq):
            k, v = K[pages, h // (Hq // Hkv), slots], V[pages, h // (Hq // Hkv), slots]
            w = np.exp(s * (k @ Q[b, h]) - wl[b, h])
            d = (Dqk + 4) * 2.0**-22 * s * (np.abs(k) @ np.abs(Q[b, h])).max()
            tol = u * np.abs(want[b, h]) + (2 * d + 2.0**-15) * (w @ np.abs(v)) + 1e-30
            if o.dtype == HF:
                tol += n * 2.0**-25 * np.abs(v).max() + 2.0**-25
            e = np.abs(O[b, h] - want[b, h])
            assert (e <= tol).all(), f"O of {b}, {h}: {e.max():.3e}, {np.max(e - tol):.3e} over its bound"
            assert abs(L[b, h] - wl[b, h]) <= d + (n + 8) * 2.0**-24 + 2.0**-21 * abs(wl[b, h]), f"LSE of {b}, {h}"


EDGES = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300, 0]
DIMS = [(64, 64), (128, 128), (128, 64), (64, 128), (256, 256), (256, 64), (64, 256), (16, 32), (32, 16), (128, 256)]


@pytest.mark.parametrize("dims", DIMS)
@pytest.mark.parametrize("dt", [BF, HF])
def test_decode_dims_and_edge_lengths(dims, dt):
    pool = Pool(EDGES, 2, *dims, 16, dt, seed=sum(dims))
    q = randn((len(EDGES), 6, dims[0]), dt, 4, 1.5)
    q[0] = float("nan")  # of an idle place: not read
    o, lse = binding.attn_paged_decode(pool.cache, q)
    q[0] = 0
    check_decode(pool, q, o, lse)
    assert binding.sync_check() == 0


@pytest.mark.parametrize("group", [1, 2, 3, 5, 8, 15, 16, 17, 31, 32, 33, 48, 64, 65, 130])
def test_decode_head_groups(group):
    pool = Pool([70, 1, 200], 2, 128, 128, 32, BF, seed=group, head_major=False)
    q = randn((3, 2 * group, 128), BF, group)
    check_decode(pool, q, *binding.attn_paged_decode(pool.cache, q))


@pytest.mark.parametrize("group,dims", [(20, (256, 256)), (40, (256, 128)), (64, (64, 256)), (40, (64, 64)), (24, (32, 128))])
def test_decode_wide_groups_and_dims(group, dims):
    pool = Pool([130, 500], 1, *dims, 64, HF, seed=group)
    q = randn((2, group, dims[0]), HF, group)
    check_decode(pool, q, *binding.attn_paged_decode(pool.cache, q))


@pytest.mark.parametrize("page", [1, 3, 8, 24, 64, 100, 256])
@pytest.mark.parametrize("head_major", [True, False])
def test_decode_pages(page, head_major):
    pool = Pool([257, 64, 5, 1000], 3, 64, 64, page, BF, seed=page, head_major=head_major)
    q = randn((4, 3, 64), BF, page)
    check_decode(pool, q, *binding.attn_paged_decode(pool.cache, q))


@pytest.mark.parametrize("B,Hkv,lens", [(1, 1, "long"), (1, 4, "long"), (3, 2, "mixed"), (200, 1, "short"), (150, 8, "one"),
                                        (400, 2, "random")])
def test_decode_splits(B, Hkv, lens):
    # one sequence over all CTAs; many sequences in one CTA; units that end in the middle of a CTA's range
    r = np.random.RandomState(B)
    n = {"long": [20011], "mixed": [9000, 1, 700], "short": list(r.randint(1, 65, B)), "one": [1] * B,
         "random": list(r.randint(0, 200, B))}[lens]
    pool = Pool([int(x) for x in n], Hkv, 64, 64, 64, BF, seed=B)
    q = randn((B, 2 * Hkv, 64), BF, B)
    o, lse = binding.attn_paged_decode(pool.cache, q)
    check_decode(pool, q, o, lse)
    o2, lse2 = binding.attn_paged_decode(pool.cache, q)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_decode_scale_sharp_scores_and_strided_q():
    pool = Pool([300, 40, 1], 2, 128, 128, 16, BF, seed=3, std=2.0)
    packed = randn((3, 9, 128), BF, 9, 3.0)
    q = packed[:, 1:5]
    check_decode(pool, q, *binding.attn_paged_decode(pool.cache, q, sm_scale=0.3), sm_scale=0.3)


def test_decode_scores_of_minus_infinity():
    # keys whose score is -inf weigh nothing; a row of nothing else is empty
    pool = Pool([130, 70], 1, 64, 64, 64, BF, seed=1)
    q = randn((2, 1, 64), BF, 2).abs_() + 0.125
    pool.k[pool.table[0, 0].item(), 0, 3:60] = float("-inf")
    for j in range(2):
        pool.k[pool.table[1, j].item()] = float("-inf")
    o, lse = binding.attn_paged_decode(pool.cache, q)
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()
    keep = [i for i in range(130) if not 3 <= i < 60]
    z = np.array([f64(pool.k[pool.table[0, i // 64].item(), 0, i % 64]) @ f64(q[0, 0]) / 8 for i in keep])
    w = np.exp(z - z.max())
    v = np.array([f64(pool.v[pool.table[0, i // 64].item(), 0, i % 64]) for i in keep])
    want = w @ v / w.sum()
    assert np.abs(f64(o[0, 0]) - want).max() <= 2.0**-8 * np.abs(want).max() + 2.0**-12 * np.abs(v).max()
    assert abs(float(lse[0, 0]) - z.max() - math.log(w.sum())) < 1e-4


def test_decode_bad_pages_and_lengths_are_reported():
    lens = [100, 64, 30]
    pool = Pool(lens, 1, 64, 64, 16, BF, seed=5)
    q = randn((3, 2, 64), BF, 5)
    good = binding.attn_paged_decode(pool.cache, q)
    for bad in (-1, pool.k.shape[0], 2**31 - 1):
        pool.table[0, 2] = bad
        o, lse = binding.attn_paged_decode(pool.cache, q)
        assert binding.sync_check() == 6
        assert binding.sync_check() == 0
        assert torch.equal(o[1:], good[0][1:]) and torch.isfinite(o).all()
    pool = Pool(lens, 1, 64, 64, 16, BF, seed=5, extra=0)
    full = pool.table.shape[1] * 16
    pool.seq_lens[1] = -5
    o, lse = binding.attn_paged_decode(pool.cache, q)
    assert binding.sync_check() == 6
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()
    pool.seq_lens[1] = 64
    pool.seq_lens[0] = full + 1000  # counts as the whole row of the table
    binding.attn_paged_decode(pool.cache, q)
    assert binding.sync_check() == 6


def test_decode_writes_its_outputs_only():
    pool = Pool([100, 0, 3], 2, 64, 64, 16, HF, seed=6)
    q = randn((3, 4, 64), HF, 6)
    ob = torch.full((3 * 4 * 64 + 128,), 7.0, dtype=HF, device="cuda")
    lb = torch.full((3 * 4 + 8,), 7.0, device="cuda")
    o, lse = ob[64:-64].view(3, 4, 64), lb[4:-4].view(3, 4)
    binding.attn_paged_decode(pool.cache, q, out=(o, lse))
    check_decode(pool, q, o, lse)
    assert (ob[:64] == 7).all() and (ob[-64:] == 7).all() and (lb[:4] == 7).all() and (lb[-4:] == 7).all()


# ------------------------------------------------------------------- append
@pytest.mark.parametrize("page,head_major", [(1, True), (5, False), (16, True), (64, False)])
@pytest.mark.parametrize("rot,inter,dims,dt", [(64, False, (64, 64), BF), (32, True, (128, 64), HF), (0, False, (64, 128), BF),
                                               (6, True, (16, 32), BF), (256, False, (256, 256), HF)])
@pytest.mark.parametrize("jagged", [False, True])
def test_append(page, head_major, rot, inter, dims, dt, jagged):
    Dqk, Dv = dims
    lens = [0, 1, 7, 64, 65, 130, 33]
    new = [0, 1, 7, 3, 0, 100, 2] if jagged else [1] * len(lens)
    pool = Pool(lens, 2, Dqk, Dv, page, dt, seed=page + rot, head_major=head_major)
    r = binding.Rope(rot, interleaved=inter, base=100.0) if rot else None
    T = sum(new) + (5 if jagged else 0)  # rows behind the last sequence
    k, v, q = (randn((T, h, d), dt, h + d) for h, d in ((2, Dqk), (2, Dv), (6, Dqk)))
    kb, vb = pool.k.clone(), pool.v.clone()
    out = torch.full_like(q, 9.0)
    off = torch.tensor([0] + new).cumsum(0).int().cuda() if jagged else None
    got = binding.attn_paged_append(pool.cache, k, v, rope=r, q=q, offsets=off, out=out)
    assert got is out and binding.sync_check() == 0
    K, V, table = pool.k.clone(), pool.v.clone(), pool.table.cpu()
    t = 0
    for b, m in enumerate(new):
        for j in range(m):
            p = lens[b] - m + j
            if p < 0:
                assert (out[t] == 0).all()  # idle
            else:
                pg, sl = int(table[b, p // page]), p % page
                for y, x in ((K[pg, :, sl], k[t]), (out[t], q[t])):
                    if r is None:
                        assert torch.equal(y, x)
                    else:
                        check_rope(y[:, None], x[:, None], [p], r)
                assert torch.equal(V[pg, :, sl], v[t])
                K[pg, :, sl], V[pg, :, sl] = kb[pg, :, sl], vb[pg, :, sl]
            t += 1
    assert same_bits(K, kb) and same_bits(V, vb)  # everything else as it was
    assert (out[t:] == 9).all()


def test_append_strided_in_place_and_without_q():
    pool = Pool([40, 3], 2, 64, 64, 16, BF, seed=1)
    r = binding.Rope(64)
    packed = randn((2, 10, 64), BF, 1)
    q, k, v = packed[:, :6], packed[:, 6:8], packed[:, 8:]
    before = packed.clone()
    a = binding.attn_paged_append(pool.cache, k, v, rope=r, q=q)
    kc = pool.k.clone()
    assert torch.equal(packed, before)
    b = binding.attn_paged_append(pool.cache, k, v, rope=r, q=q, out=q)
    assert b is q and torch.equal(a, packed[:, :6]) and torch.equal(packed[:, 6:], before[:, 6:])
    assert binding.attn_paged_append(pool.cache, k, v, rope=r) is None
    assert same_bits(kc, pool.k)
    # jagged [H, T, D] tensors, as the attention kernels take them
    kj, vj = k.transpose(0, 1).contiguous(), v.transpose(0, 1).contiguous()
    binding.attn_paged_append(pool.cache, kj.transpose(0, 1), vj.transpose(0, 1), rope=r)
    assert same_bits(kc, pool.k)
    # rows off 16-byte boundaries
    buf = torch.empty((2, 2, 64 + 3), dtype=BF, device="cuda")
    buf[..., 3:] = k
    binding.attn_paged_append(pool.cache, buf[..., 3:], v, rope=r)
    assert same_bits(kc, pool.k)


@pytest.mark.parametrize("what", ["page", "table", "length"])
def test_append_bad_places_are_reported_and_left_out(what):
    r = binding.Rope(64)
    k, v, q = randn((2, 1, 64), BF, 1), randn((2, 1, 64), BF, 2), randn((2, 2, 64), BF, 3)
    pool = Pool([40, 3], 1, 64, 64, 16, BF, seed=2, extra=0)
    off = None
    if what == "page":
        pool.table[0, 2] = pool.k.shape[0]
    elif what == "table":
        pool.seq_lens[0] = 16 * pool.table.shape[1] + 1
    else:
        pool.seq_lens[0] = 1  # two tokens, one place
        off = torch.tensor([0, 2, 2], dtype=torch.int32).cuda()
    kb, vb = pool.k.clone(), pool.v.clone()
    y = binding.attn_paged_append(pool.cache, k, v, rope=r, q=q, offsets=off)
    assert binding.sync_check() == 6 and binding.sync_check() == 0
    if what == "length":
        assert (y[0] == 0).all()
        check_rope(y[1][:, None], q[1][:, None], [0], r)
        p, slot = int(pool.table[0, 0]), 0
    else:
        p, slot = int(pool.table[1, 0]), 2
    assert torch.equal(pool.v[p, :, slot], v[1])
    pool.k[p, :, slot], pool.v[p, :, slot] = kb[p, :, slot], vb[p, :, slot]
    assert same_bits(pool.k, kb) and same_bits(pool.v, vb)


def test_cache_refusals():
    pool = Pool([40, 3], 2, 64, 64, 16, BF)
    c, q, k = pool.cache, randn((2, 4, 64), BF, 0), randn((2, 2, 64), BF, 1)
    for bad in (lambda: binding.attn_paged_decode(c, q[:1]), lambda: binding.attn_paged_decode(c, q[:, :3]),
                lambda: binding.attn_paged_decode(c, q.cpu()), lambda: binding.attn_paged_decode(c, q[..., :32]),
                lambda: binding.attn_paged_decode(c, q, out=(q[:, :2], torch.empty(2, 4, device="cuda"))),
                lambda: binding.attn_paged_append(c, k[:1], k[:1]), lambda: binding.attn_paged_append(c, k, k[:, :1]),
                lambda: binding.attn_paged_append(c, k, k, q=q[..., :32]), lambda: binding.attn_paged_append(c, k, k, out=q),
                lambda: binding.attn_paged_append(c, k, k, q=q, out=q[:, :2]),
                lambda: binding.attn_paged_append(c, k, k, rope=binding.Rope(128)),
                lambda: binding.attn_paged_append(c, k, k, offsets=torch.zeros(2, dtype=torch.int32, device="cuda")),
                lambda: binding.PagedCache(pool.k, pool.v, pool.table[0], pool.seq_lens),
                lambda: binding.PagedCache(pool.k, pool.v[:1], pool.table, pool.seq_lens),
                lambda: binding.PagedCache(pool.k, pool.v, pool.table, pool.seq_lens[:1]),
                lambda: binding.PagedCache(pool.k.transpose(2, 3), pool.v, pool.table, pool.seq_lens)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: binding.attn_paged_decode(c, q.half()), lambda: binding.attn_paged_append(c, k, k.float()),
                lambda: binding.PagedCache(pool.k, pool.v.half(), pool.table, pool.seq_lens),
                lambda: binding.PagedCache(pool.k, pool.v, pool.table.long(), pool.seq_lens)):
        with pytest.raises(TypeError):
            bad()
    wide = torch.zeros((2, 2, 16, 96), dtype=BF, device="cuda")
    with pytest.raises(binding.AttnError):
        binding.attn_paged_decode(binding.PagedCache(wide, wide, pool.table, pool.seq_lens), torch.zeros(2, 2, 96, dtype=BF, device="cuda"))
    odd = torch.zeros((2, 2, 16, 68), dtype=BF, device="cuda")[..., :64]
    with pytest.raises(binding.AttnError):
        binding.attn_paged_decode(binding.PagedCache(odd, odd, pool.table, pool.seq_lens), q)


def test_nothing_to_do():
    r = binding.Rope(64)
    x = torch.empty((2, 0, 4, 64), dtype=BF, device="cuda")
    assert binding.attn_rope([x, x], r)[0].shape == x.shape
    assert binding.attn_rope([x.view(0, 8, 64)], r, offsets=torch.tensor([0, 8], dtype=torch.int32).cuda())[0].numel() == 0
    pool = Pool([0, 0], 2, 64, 64, 16, BF)
    q, k = randn((2, 4, 64), BF, 0), randn((2, 2, 64), BF, 1)
    kb = pool.k.clone()
    y = binding.attn_paged_append(pool.cache, k, k, rope=r, q=q)
    assert (y == 0).all() and same_bits(kb, pool.k)
    o, lse = binding.attn_paged_decode(pool.cache, q)
    assert (o == 0).all() and torch.isneginf(lse).all()
    empty = binding.PagedCache(pool.k, pool.v, pool.table[:0], pool.seq_lens[:0])
    assert binding.attn_paged_decode(empty, q[:0])[0].shape == (0, 4, 64)
    assert binding.attn_paged_append(empty, k[:0], k[:0]) is None
    assert binding.sync_check() == 0


# ----------------------------------------------------------------- together
@pytest.mark.parametrize("dims,inter,dt", [((64, 64), False, BF), ((128, 64), True, HF)])
def test_prompt_then_tokens_equals_one_causal_attention(dims, inter, dt):
    """A program that serves: rotate and attend over the prompts, put them in
    the cache, then token by token append and decode; every row of every
    sequence against the float64 causal attention over the whole of it."""
    Dqk, Dv = dims
    H, steps, page = 3, 6, 16
    prompt = [70, 1, 33]
    total = [n + steps for n in prompt]
    r = binding.Rope(Dqk, interleaved=inter, scaling="linear", factor=2.0)
    full = [[randn((H, n, d), dt, 31 * i + j) for j, d in enumerate((Dqk, Dqk, Dv))] for i, n in enumerate(total)]
    # prompts, packed [H, T, D]
    q, k, v = (torch.cat([full[i][j][:, :n] for i, n in enumerate(prompt)], 1).contiguous() for j in range(3))
    off = torch.tensor([0] + prompt).cumsum(0).int().cuda()
    qr, kr = binding.attn_rope([q, k], r, offsets=off)
    o, _ = binding.attn_fwd(qr, kr, v, causal=True, offsets=off, max_seq_len=max(prompt))
    rows = [[o[:, off[i]:off[i + 1]]] for i in range(3)]
    # the cache
    per = [-(-n // page) for n in total]
    pools = [torch.full((sum(per) + 1, H, page, d), float("nan"), dtype=dt, device="cuda") for d in dims]
    table = torch.zeros((3, max(per)), dtype=torch.int32)
    ids = torch.randperm(sum(per) + 1, generator=torch.Generator().manual_seed(1))
    for i in range(3):
        table[i, :per[i]] = ids[sum(per[:i]):sum(per[:i + 1])].int()
    lens = torch.tensor(prompt, dtype=torch.int32).cuda()
    cache = binding.PagedCache(*pools, table.cuda(), lens)
    binding.attn_paged_append(cache, k.transpose(0, 1), v.transpose(0, 1), rope=r, offsets=off)
    # the keys in the cache are the rotated ones, bit for bit
    for i, n in enumerate(prompt):
        got = torch.cat([pools[0][int(table[i, j])] for j in range(per[i])], 1)[:, :n]
        assert torch.equal(got, kr[:, off[i]:off[i + 1]])
    for s in range(steps):
        lens += 1
        qt, kt, vt = (torch.stack([full[i][j][:, prompt[i] + s] for i in range(3)]) for j in range(3))
        qt = binding.attn_paged_append(cache, kt, vt, rope=r, q=qt)
        o, _ = binding.attn_paged_decode(cache, qt)
        for i in range(3):
            rows[i].append(o[i][:, None])
    assert binding.sync_check() == 0
    for i in range(3):
        a = [f64(t) for t in full[i]]
        w = f64(r.inv_freq)
        a[0], a[1] = (paged_ref.rope(x, range(total[i]), w, inter) for x in a[:2])
        want = oracle.attention_fwd(a[0][None], a[1][None], a[2][None], causal=True)[0][0]
        got = f64(torch.cat(rows[i], 1))
        # the attention's bar, and the 16-bit rounding of the rotated q and k:
        # each moves a score by at most u sum |q||k| s
        u = torch.finfo(dt).eps / 2
        d = 2 * u * Dqk**-0.5 * np.einsum("hid,hjd->hij", np.abs(a[0]), np.abs(a[1])).max()
        assert np.abs(got - want).max() <= 1e-2 + 2 * d * np.abs(a[2]).max()


def test_rotated_jvp_and_backward():
    """Training with tangents: q, k, tq, tk rotated in one launch, forward +
    JVP, the backward, dq and dk turned back; against the float64 oracle of
    the unrotated inputs (rotated in 64 bits)."""
    B, H, N, D = 1, 2, 100, 64
    r = binding.Rope(32, interleaved=True)
    q, k, v, tq, tk, tv, do = (randn((B, H, N, D), BF, s, 0.5) for s in range(7))
    qr, kr, tqr, tkr = binding.attn_rope([q, k, tq, tk], r)
    o, to, lse = binding.attn_fwd_jvp(qr, kr, v, tqr, tkr, tv, causal=True)
    dq, dk, dv, _ = binding.attn_bwd(qr, kr, v, o, lse, do, causal=True)
    dq, dk = binding.attn_rope([dq, dk], r, inverse=True)
    assert binding.sync_check() == 0
    w, pos = f64(r.inv_freq), range(N)
    rot = lambda x, **kw: paged_ref.rope(f64(x) if torch.is_tensor(x) else x, pos, w, True, **kw)  # noqa: E731
    O, tO, _ = oracle.attention_fwd_jvp(rot(q), rot(k), f64(v), rot(tq), rot(tk), f64(tv), causal=True)
    g = oracle.attention_bwd(rot(q), rot(k), f64(v), f64(do), causal=True)
    for got, want in ((o, O), (to, tO), (dq, rot(g[0], inverse=True)), (dk, rot(g[1], inverse=True)), (dv, g[2])):
        assert np.abs(f64(got) - want).max() <= 2e-2 * max(1.0, np.abs(want).max())


def test_captured_step_replays_with_new_lengths():
    pool = Pool([64, 1, 200], 2, 64, 64, 16, BF, seed=4, extra=4)
    # room to grow: pages of their own behind the pool
    more = torch.zeros((12, 2, 16, 64), dtype=BF, device="cuda")
    k, v = torch.cat([pool.k, more]), torch.cat([pool.v, more])
    table = pool.table.clone()
    for b, n in enumerate(pool.lens):
        j = -(-n // 16)
        table[b, j:j + 4] = torch.arange(4, device="cuda", dtype=torch.int32) + pool.k.shape[0] + 4 * b
    lens = pool.seq_lens.clone()
    cache, r = binding.PagedCache(k, v, table, lens), binding.Rope(64)
    q, kn, vn = randn((3, 4, 64), BF, 1), randn((3, 2, 64), BF, 2), randn((3, 2, 64), BF, 3)

    def step():
        lens.add_(1)
        return binding.attn_paged_decode(cache, binding.attn_paged_append(cache, kn, vn, rope=r, q=q))

    k0, v0, l0 = k.clone(), v.clone(), lens.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    got = []
    for replay in (True, False):
        k.copy_(k0), v.copy_(v0), lens.copy_(l0)
        for i in range(20):
            if i == 10:
                lens[1] = -1  # the second place is idle in this step, and starts anew behind it
            q.copy_(randn((3, 4, 64), BF, 50 + i))
            if replay:
                graph.replay()
                got.append((o.clone(), lse.clone()))
                assert i != 10 or (o[1] == 0).all()
            else:
                a, b = step()
                assert torch.equal(a, got[i][0]) and torch.equal(b, got[i][1]), i
    assert binding.sync_check() == 0


def test_first_call_may_be_captured():
    """In a process of its own: the first calls of the library are captured."""
    import os
    import subprocess
    import sys
    code = """
import torch
from attention_forward_jvp_gb300 import binding
t = lambda *s: torch.ones(s, dtype=torch.bfloat16, device="cuda")
k, v, q, kn = t(4, 2, 16, 64), t(4, 2, 16, 64), t(2, 4, 64), t(2, 2, 64)
cache = binding.PagedCache(k, v, torch.arange(4, device="cuda", dtype=torch.int32).view(2, 2),
                           torch.tensor([20, 3], device="cuda", dtype=torch.int32))
r = binding.Rope(64)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    x = binding.attn_rope([q[None]], r)[0]
    o, lse = binding.attn_paged_decode(cache, binding.attn_paged_append(cache, kn, kn, rope=r, q=q))
g.replay()
torch.cuda.synchronize()
assert (o == 1).all() and torch.isfinite(lse).all() and torch.equal(x[:, :1, 0], q[None][:, :1, 0])
assert binding.sync_check() == 0
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def test_calls_on_two_streams_and_two_graphs_at_once():
    pools = [Pool([20000, 300], 2, 64, 64, 64, BF, seed=s) for s in (1, 2)]
    qs = [randn((2, 8, 64), BF, s) for s in (3, 4)]
    want = [binding.attn_paged_decode(p.cache, q) for p, q in zip(pools, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(binding.attn_paged_decode(pools[i].cache, qs[i]))
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):  # captured on one stream, replayed on two
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=streams[0]):
            out = binding.attn_paged_decode(pools[i].cache, qs[i])
        graphs.append((g, out))
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                graphs[i][0].replay()
    torch.cuda.synchronize()
    for i in range(2):
        got[i].append(graphs[i][1])
        for o, lse in got[i]:
            assert torch.equal(o, want[i][0]) and torch.equal(lse, want[i][1])


def test_inputs_written_just_before_the_call_are_seen():
    # every kernel here is launched before the one ahead of it has ended
    pool = Pool([500, 64], 2, 64, 64, 64, BF, seed=9)
    r = binding.Rope(64)
    a, k, v = randn((2, 4, 64), BF, 1), randn((2, 2, 64), BF, 2), randn((2, 2, 64), BF, 3)
    q, kc = torch.empty_like(a), pool.k.clone()
    outs = []
    for wait in (True, False):
        pool.k.copy_(kc)
        for i in range(30):
            for x in (lambda: q.copy_(a * (1 + i % 3)),
                      lambda: binding.attn_paged_append(pool.cache, k * (i + 1), v, rope=r, q=q, out=q),
                      lambda: outs.append(binding.attn_paged_decode(pool.cache, q))):
                x()
                if wait:
                    torch.cuda.synchronize()
    torch.cuda.synchronize()
    for (o, lse), (o2, lse2) in zip(outs[:30], outs[30:]):
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_launch_counts():
    pool = Pool([40, 3], 2, 64, 64, 16, BF)
    q, k, r = randn((2, 4, 64), BF, 0), randn((2, 2, 64), BF, 1), binding.Rope(64)
    n = binding.launch_count()
    binding.attn_rope([q[None], q[None], q[None]], r)
    binding.attn_paged_append(pool.cache, k, k, rope=r, q=q)
    assert binding.launch_count() == n + 2


def test_pool_offsets_pass_32_bits():
    # a pool of more than 2^31 elements, pages at both of its ends
    page, H, D = 64, 2, 128
    n_pages = (1 << 31) // (page * H * D) + 200
    k = torch.zeros((n_pages, H, page, D), dtype=BF, device="cuda")
    v = torch.zeros((n_pages, H, page, D), dtype=BF, device="cuda")
    ids = [0, n_pages - 1, n_pages - 150, 3]
    table, lens = torch.tensor([ids], dtype=torch.int32).cuda(), torch.tensor([250], dtype=torch.int32).cuda()
    kn, vn = randn((250, H, D), BF, 1), randn((250, H, D), BF, 2)
    cache = binding.PagedCache(k, v, table, lens)
    binding.attn_paged_append(cache, kn, vn, offsets=torch.tensor([0, 250], dtype=torch.int32).cuda())
    q = randn((1, 8, D), BF, 3)
    o, lse = binding.attn_paged_decode(cache, q)
    small = Pool([250], H, D, D, page, BF)
    for j in range(4):
        m = min(page, 250 - j * page)
        p = int(small.table[0, j])
        small.k[p, :, :m] = kn[j * page:j * page + m].transpose(0, 1)
        small.v[p, :, :m] = vn[j * page:j * page + m].transpose(0, 1)
        assert torch.equal(k[ids[j], :, :m], small.k[p, :, :m]) and torch.equal(v[ids[j], :, :m], small.v[p, :, :m])
    check_decode(small, q, o, lse)
    assert binding.sync_check() == 0


def test_decode_wait_that_runs_out_is_reported():
    # many heads: the kernel whose warps wait for one another.  A first tile
    # that never arrives (host-set hook) ends every wait within its bound; the
    # context and the next call are sound.
    pool = Pool([300, 70], 1, 128, 64, 16, BF, seed=8)
    q = randn((2, 40, 128), BF, 8)
    binding.set_wait_timeout_ns(20_000_000)
    binding.debug_skip_first_load(True)
    try:
        binding.attn_paged_decode(pool.cache, q)
        assert binding.sync_check() == 5
    finally:
        binding.debug_skip_first_load(False)
        binding.set_wait_timeout_ns(2_000_000_000)
    assert binding.sync_check() == 0
    check_decode(pool, q, *binding.attn_paged_decode(pool.cache, q))


@pytest.mark.parametrize("B,Hkv,group,lens", [(1, 1, 64, "long"), (2, 1, 17, "mixed"), (40, 2, 33, "short"),
                                              (30, 3, 100, "random"), (1, 2, 128, "long")])
def test_decode_many_heads_splits(B, Hkv, group, lens):
    r = np.random.RandomState(B + group)
    n = {"long": [9011], "mixed": [5000, 130], "short": list(r.randint(1, 65, B)), "random": list(r.randint(0, 400, B))}[lens]
    pool = Pool([int(x) for x in n], Hkv, 64, 64, 32, HF if group == 33 else BF, seed=B)
    q = randn((B, group * Hkv, 64), pool.k.dtype, B, 2.0)
    o, lse = binding.attn_paged_decode(pool.cache, q)
    check_decode(pool, q, o, lse)
    o2, lse2 = binding.attn_paged_decode(pool.cache, q)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dims,group", [((256, 256), 12), ((256, 256), 70), ((64, 64), 20)])
@pytest.mark.parametrize("lens", ["one tile", "random"])
def test_decode_many_short_sequences(dims, group, lens):
    # a CTA's units change with every tile or two (both head dims 256: each group of producers skips some), and
    # there are more sequences than a CTA has threads
    r = np.random.RandomState(group)
    B = 700
    n = list(r.randint(1, 65, B)) if lens == "one tile" else list(r.randint(0, 200, B))
    pool = Pool([int(x) for x in n], 2, *dims, 16, BF, seed=group)
    q = randn((B, 2 * group, dims[0]), BF, group)
    o, lse = binding.attn_paged_decode(pool.cache, q)
    check_decode(pool, q, o, lse)
    o2, lse2 = binding.attn_paged_decode(pool.cache, q)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("D,rot", [(96, 96), (48, 32), (80, 40)])
def test_rope_jagged_rows_that_do_not_fill_a_block(D, rot):
    # threads behind a block's last row; more sequences than a warp's search takes at once
    r = np.random.RandomState(D)
    lens = [int(x) for x in r.randint(0, 4, 1500)]
    T = sum(lens)
    off = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    x = randn((2, T, D), BF, D)
    rope = binding.Rope(rot)
    (y,) = binding.attn_rope([x], rope, offsets=off)
    pos = torch.tensor(np.concatenate([np.arange(n) for n in lens]), dtype=torch.int32, device="cuda")
    (z,) = binding.attn_rope([x[None]], rope, positions=pos)
    assert torch.equal(y, z[0])


@pytest.mark.parametrize("group", [4, 40])
@pytest.mark.parametrize("bad", ["nan key", "nan value", "inf value"])
def test_decode_nonfinite_entries_stay_with_their_key_head(group, bad):
    pool = Pool([200, 90], 2, 64, 64, 16, BF, seed=group)
    q = randn((2, 2 * group, 64), BF, group)
    o, lse = binding.attn_paged_decode(pool.cache, q)
    page = int(pool.table[0, 3])  # sequence 0, tokens 48 .. 63
    x = pool.k if bad == "nan key" else pool.v
    x[page, 1, 5, 7] = float("inf") if bad == "inf value" else float("nan")
    o2, lse2 = binding.attn_paged_decode(pool.cache, q)
    assert torch.equal(o[1], o2[1]) and torch.equal(o[0, :group], o2[0, :group])
    assert torch.equal(lse[1], lse2[1]) and torch.equal(lse[0, :group], lse2[0, :group])
    if bad == "nan key":
        assert torch.isnan(o2[0, group:]).all() and torch.isnan(lse2[0, group:]).all()
    else:
        hit = torch.arange(64, device="cuda") == 7
        # a probability is the sum of two parts, and the second may have any sign: infinity or NaN
        assert (torch.isnan(o2[0, group:, hit]) | (torch.isinf(o2[0, group:, hit]) & (bad == "inf value"))).all()
        assert torch.equal(o2[0, group:][:, ~hit], o[0, group:][:, ~hit])
        assert torch.equal(lse, lse2)


@pytest.mark.parametrize("group", [2, 20])
def test_decode_of_a_table_whose_steps_pass_31_bits(group):
    # the rows of the table are as long as the struct says only where a length reaches: planned in 64 bits, the
    # same ranges and results
    r = np.random.RandomState(group)
    pool = Pool([int(x) for x in r.randint(0, 300, 40)], 2, 64, 64, 16, BF, seed=group)
    q = randn((40, 2 * group, 64), BF, group)
    o, lse = binding.attn_paged_decode(pool.cache, q)
    pool.cache._struct.max_pages = 1 << 26
    o2, lse2 = binding.attn_paged_decode(pool.cache, q)
    check_decode(pool, q, o2, lse2)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("group", [2, 20])
def test_decode_of_an_empty_pool(group):
    k = torch.empty((0, 2, 16, 64), dtype=BF, device="cuda")
    table, lens = torch.zeros((3, 4), dtype=torch.int32, device="cuda"), [50, 0, 7]
    cache = binding.PagedCache(k, k, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    o, lse = binding.attn_paged_decode(cache, randn((3, 2 * group, 64), BF, 0))
    assert binding.sync_check() == 6
    assert (o == 0).all()
    for b, n in enumerate(lens):  # keys of zero: every score is 0
        want = np.log(n) if n else -np.inf
        assert (f64(lse[b]) == want).all() if n == 0 else (np.abs(f64(lse[b]) - want) <= 2.0**-20).all()


@pytest.mark.parametrize("dims,group", [((64, 64), 24), ((64, 64), 32), ((128, 64), 30), ((256, 64), 23), ((64, 128), 20),
                                        ((128, 128), 24), ((32, 16), 29), ((16, 128), 18)])
@pytest.mark.parametrize("page", [16, 24])
def test_decode_three_and_four_groups_of_heads(dims, group, page):
    # lengths about the ends of steps and ranges, one long one; pages of whole steps and not
    pool = Pool([1, 16, 17, 0, 63, 300, 5000], 2, *dims, page, HF, seed=group + page)
    q = randn((7, 2 * group, dims[0]), HF, group, 1.5)
    o, lse = binding.attn_paged_decode(pool.cache, q)
    check_decode(pool, q, o, lse)
    o2, lse2 = binding.attn_paged_decode(pool.cache, q)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_decode_of_sequences_that_share_pages():
    pool = Pool([200, 90, 33], 2, 64, 64, 16, BF, seed=1)
    pool.table[1] = pool.table[0]
    pool.table[2, :2] = pool.table[0, :2]
    pool.table[2, 2] = pool.table[0, 2]
    for group in (3, 40):
        q = randn((3, 2 * group, 64), BF, group)
        check_decode(pool, q, *binding.attn_paged_decode(pool.cache, q))


@pytest.mark.parametrize("lens,Hkv", [([5], 1), ([77], 2), ([33, 0, 48], 1), ([112], 1), ([128], 2), ([0], 2)])
def test_decode_of_lists_about_as_long_as_one_block_holds(lens, Hkv):
    pool = Pool(lens, Hkv, 128, 64, 16, BF, seed=len(lens), extra=0)
    q = randn((len(lens), 5 * Hkv, 128), BF, 3)
    check_decode(pool, q, *binding.attn_paged_decode(pool.cache, q))
