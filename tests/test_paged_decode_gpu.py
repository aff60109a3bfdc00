"""Paged decode on the GPU where its arithmetic and its refusals are thinnest,
against the float64 definition of oracle.paged_ref.

Tolerances, from the arithmetic (u = half a step of the output type,
torch.finfo(t).eps / 2):

  scores   d = (Dqk + 4) 2^-22 s max_j sum |q| |k_j|: fp32 sums, a rounding
           and a truncation each
  O        u |O| + (2 d + 2^-15) sum_j w_j |V_j|: a weight is off by its own
           score's error and the others', by exp2's (2^-22) and by what P's
           two parts leave (bf16 2^-18, fp16 2^-22 of it), and the sum by its
           accumulation
  LSE      d + (n + 8) 2^-24 + 2^-21 |LSE|
"""
import numpy as np
import pytest
import torch

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
    return (torch.randn(shape, generator=g) * std).to(dtype)


class Pool:
    """Keys and values [pages, Hkv, page, d] of the CPU, a shuffled page table
    (entries behind a sequence's last page are out of range), and the cache of
    them on the GPU.  Every slot of every page is finite."""

    def __init__(self, lens, Hkv, Dqk, Dv, page, dtype, seed=0, width=None):
        need = [-(-n // page) for n in lens]
        width = width or max(need + [1])
        self.lens, self.page, count = list(lens), page, sum(need) + 2
        self.k, self.v = (randn((count, Hkv, page, d), dtype, seed + i) for i, d in enumerate((Dqk, Dv)))
        order = torch.randperm(count, generator=torch.Generator().manual_seed(seed))
        self.table = torch.full((len(lens), width), -7, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n].int()
            at += n

    def rows(self, x, b, h):
        """Rows of a pool's key head in the order of sequence b."""
        j = torch.arange(self.lens[b])
        return x[self.table[b, j // self.page].long(), h, j % self.page]

    def cache(self, table=None, lens=None):
        table = self.table if table is None else table
        lens = torch.tensor(self.lens if lens is None else lens, dtype=torch.int32)
        return binding.PagedCache(self.k.cuda(), self.v.cuda(), table.cuda(), lens.cuda())


def check(pool, q, o, lse, sm_scale=None):
    Q, K, V = f64(q), f64(pool.k), f64(pool.v)
    want, wl = paged_ref.decode(Q, K, V, pool.table.numpy(), pool.lens, sm_scale)
    O, L, u = f64(o), f64(lse), torch.finfo(o.dtype).eps / 2
    group, Dqk = Q.shape[1] // K.shape[1], Q.shape[2]
    s = Dqk**-0.5 if sm_scale is None else sm_scale
    assert np.isfinite(O).all() and not np.isnan(L).any()
    for b, n in enumerate(pool.lens):
        if n == 0:
            assert (O[b] == 0).all() and np.isneginf(L[b]).all()
            continue
        for h in range(Q.shape[1]):
            k, v = f64(pool.rows(pool.k, b, h // group)), f64(pool.rows(pool.v, b, h // group))
            w = np.exp(s * (k @ Q[b, h]) - wl[b, h])
            d = (Dqk + 4) * 2.0**-22 * s * (np.abs(k) @ np.abs(Q[b, h])).max()
            tol = u * np.abs(want[b, h]) + (2 * d + 2.0**-15) * (w @ np.abs(v))
            tol += torch.finfo(o.dtype).smallest_normal * 2 * u
            e = np.abs(O[b, h] - want[b, h])
            assert (e <= tol).all(), f"O of {b}, {h}: {e.max():.3e}, {np.max(e - tol):.3e} over its bound"
            assert abs(L[b, h] - wl[b, h]) <= d + (n + 8) * 2.0**-24 + 2.0**-21 * abs(wl[b, h]), f"LSE of {b}, {h}"


@pytest.mark.parametrize("dims", [(64, 64), (128, 128), (64, 256), (256, 128), (256, 256)])
@pytest.mark.parametrize("group", [33, 65, 95, 97, 127])
def test_heads_that_end_inside_a_quadrant(dims, group):
    # (33 stand twice, the others once; units that end in a CTA and that several share)
    pool = Pool([1, 64, 65, 0, 1500], 1, *dims, 16, BF if group % 4 == 1 else HF, seed=group)
    q = randn((5, group, dims[0]), pool.k.dtype, group)
    check(pool, q, *binding.attn_paged_decode(pool.cache(), q.cuda()))


@pytest.mark.parametrize("dims,group", [((64, 64), 1), ((64, 64), 24), ((128, 128), 8), ((256, 256), 5), ((64, 64), 40),
                                        ((128, 64), 70), ((256, 256), 12)])
@pytest.mark.parametrize("dt", [BF, HF])
def test_one_key_that_outweighs_an_even_tail(dims, group, dt):
    """In every 16 keys one of value 0 that outweighs each of the others by
    2^6 to 2^28, by the head: O is the tail's, and LSE has both.  The tail's
    weights are all alike, so that what the parts of P drop adds up.  Beside
    the module's bound only that: fp16 parts drop up to 2^-25 of a weight
    that is 2^-11 of the largest or more, each 2^-36 of the large key's."""
    Dqk, Dv = dims
    lens = [16, 64, 1000, 5, 3000]
    pool = Pool(lens, 1, Dqk, Dv, 16, dt, seed=group)
    pool.k.zero_()
    pool.k[:, :, 3, 0] = 8.0
    pool.v.copy_((torch.rand(pool.v.shape, generator=torch.Generator().manual_seed(1)) + 0.5) * 2.0**13)
    pool.v[:, :, 3] = 0.0
    q = randn((5, group, Dqk), dt, group)
    gap = torch.linspace(6.0, 28.0, group) if group > 1 else torch.tensor([24.7])
    q[:, :, 0] = (gap * np.log(2.0) * Dqk**0.5 / 8.0).to(dt)  # score of the large key over the others' 0
    o, lse = binding.attn_paged_decode(pool.cache(), q.cuda())
    u, O, L = torch.finfo(dt).eps / 2, f64(o), f64(lse)
    for b, n in enumerate(lens):
        v, big = f64(pool.rows(pool.v, b, 0)), np.arange(n) % 16 == 3
        for h in range(group):
            z = float(q[b, h, 0].double()) * 8.0 * Dqk**-0.5
            total = big.sum() * np.exp(z) + (~big).sum()
            want, d = v.sum(0) / total, (Dqk + 4) * 2.0**-22 * z
            drop = 2.0**-36 * np.exp(z) * v.sum(0) / total if dt == HF else 0.0
            tol = (u + 2 * d + 2.0**-15) * want + drop + (2.0**-25 if dt == HF else 0.0)
            e = np.abs(O[b, h] - want)
            assert (e <= tol).all(), f"O of {b}, gap 2^{z / np.log(2.0):.1f}: {np.max(e / want):.2e} of it"
            assert abs(L[b, h] - np.log(total)) <= d + (n + 8) * 2.0**-24 + 2.0**-21 * np.log(total)


def test_large_keys_that_come_late():
    # the maximum rises by 2^3 to 2^14 from one 64 keys to the next: the reference moves, and with it what was added up
    for dt in (BF, HF):
        for dims, group in (((64, 64), 3), ((64, 128), 30), ((128, 128), 70)):
            pool = Pool([700, 65, 3001], 1, *dims, 16, dt, seed=group)
            for b, n in enumerate(pool.lens):
                j = torch.arange(n)
                step = [3.0, 14.0, 0.4][b]
                pool.k[pool.table[b, j // 16].long(), 0, j % 16, 0] += (j // 64 * step).to(dt)
            q = randn((3, group, dims[0]), dt, group)
            q[:, :, 0] = dims[0] ** 0.5
            check(pool, q, *binding.attn_paged_decode(pool.cache(), q.cuda()))


def test_bad_page_beside_a_wait_that_runs_out_is_reported_next():
    # a first tile that never arrives (host-set hook), and a page out of range in it: both are told, one after the other
    pool = Pool([300, 70], 1, 128, 64, 16, BF, seed=8)
    q = randn((2, 40, 128), BF, 8).cuda()
    bad = pool.table.clone()
    bad[0, 1] = -1
    cache = pool.cache(table=bad)
    binding.set_wait_timeout_ns(20_000_000)
    binding.debug_skip_first_load(True)
    try:
        binding.attn_paged_decode(cache, q)
        assert [binding.sync_check() for _ in range(3)] == [5, 6, 0]
    finally:
        binding.debug_skip_first_load(False)
        binding.set_wait_timeout_ns(2_000_000_000)
    binding.attn_paged_decode(cache, q)
    assert [binding.sync_check() for _ in range(2)] == [6, 0]
    check(pool, q, *binding.attn_paged_decode(pool.cache(), q))


@pytest.mark.parametrize("group,dims", [(2, (64, 64)), (40, (64, 64)), (70, (128, 128)), (12, (256, 256)), (6, (16, 32))])
@pytest.mark.parametrize("page", [16, 24])
@pytest.mark.parametrize("bad", [-1, 2**31 - 1, None])
def test_bad_pages_count_as_zeros(group, dims, page, bad):
    # keys and values of zero among good ones, in a page that ends inside a step and in the last one
    pool = Pool([100, 64, 500], 2, *dims, page, HF, seed=group)
    q = randn((3, 2 * group, dims[0]), HF, group)
    table = pool.table.clone()
    for b, e in ((0, 1), (2, 4), (2, int((pool.table[2] >= 0).sum()) - 1)):
        table[b, e] = pool.k.shape[0] if bad is None else bad
        pool.k[pool.table[b, e].long()] = 0
        pool.v[pool.table[b, e].long()] = 0
    o, lse = binding.attn_paged_decode(pool.cache(table=table), q.cuda())
    assert binding.sync_check() == 6
    check(pool, q, o, lse)
    o2, lse2 = binding.attn_paged_decode(pool.cache(), q.cuda())
    assert binding.sync_check() == 0
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("group,dims", [(2, (64, 64)), (40, (64, 64)), (70, (128, 128))])
@pytest.mark.parametrize("page", [16, 24])
def test_lengths_out_of_range_count_as_the_nearer_bound(group, dims, page):
    lens = [13 * page, 50, 0]
    pool = Pool(lens, 2, *dims, page, BF, seed=group, width=13)
    q = randn((3, 2 * group, dims[0]), BF, group).cuda()
    for long in (13 * page + 1, 2**31 - 1):
        o, lse = binding.attn_paged_decode(pool.cache(lens=[long, 50, -3]), q)
        assert binding.sync_check() == 6
        check(pool, q, o, lse)


@pytest.mark.parametrize("shape", [(), (64,), (2, 64), (1, 2, 3, 4, 64)])
def test_tensors_of_other_dimensions_are_refused(shape):
    pool = Pool([40, 3], 2, 64, 64, 16, BF)
    c, r, bad = pool.cache(), binding.Rope(64), torch.zeros(shape, dtype=BF, device="cuda")
    x, q, k = (randn(s, BF, 0).cuda() for s in ((1, 2, 4, 64), (2, 4, 64), (2, 2, 64)))
    calls = [lambda: binding.attn_rope([bad], r), lambda: binding.attn_rope([x, bad], r),
             lambda: binding.attn_rope([x], r, out=[bad]), lambda: binding.attn_paged_append(c, bad, k),
             lambda: binding.attn_paged_append(c, k, bad), lambda: binding.attn_paged_append(c, k, k, q=bad),
             lambda: binding.attn_paged_append(c, k, k, q=q, out=bad), lambda: binding.attn_paged_decode(c, bad),
             lambda: binding.PagedCache(bad, c.v, c.page_table, c.seq_lens),
             lambda: binding.PagedCache(c.k, bad, c.page_table, c.seq_lens),
             lambda: binding.PagedCache(c.k, c.v, c.page_table, bad.int())]
    if bad.dim() != 2:
        calls.append(lambda: binding.PagedCache(c.k, c.v, bad.int(), c.seq_lens))
    for call in calls:
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("dims", [(64, 64), (128, 64)])
def test_one_pool_for_keys_and_values(dims):
    # values that are the first elements of the keys, in their place: written as both, read as both
    pool = Pool([40, 3], 2, dims[0], dims[1], 16, BF, seed=2)
    k, kn = pool.k.cuda(), randn((2, 2, dims[0]), BF, 1).cuda()
    c = binding.PagedCache(k, k[..., :dims[1]], pool.table.cuda(), torch.tensor(pool.lens, dtype=torch.int32).cuda())
    binding.attn_paged_append(c, kn, kn[..., :dims[1]])
    for b, n in enumerate(pool.lens):
        pool.k[pool.table[b, (n - 1) // 16].long(), :, (n - 1) % 16] = kn[b].cpu()
    assert torch.equal(k.cpu(), pool.k)
    pool.v = pool.k[..., :dims[1]]
    q = randn((2, 6, dims[0]), BF, 3)
    check(pool, q, *binding.attn_paged_decode(c, q.cuda()))
    for bad in (dict(rope=binding.Rope(64)), dict(v=kn[..., :dims[1]].clone())):
        with pytest.raises(binding.AttnError):
            binding.attn_paged_append(c, kn, bad.pop("v", kn[..., :dims[1]]), **bad)
