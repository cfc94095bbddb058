"""The attention operators (4-bit cache store / load / attend / evict, prompt attention)
against plain implementations in 64 bits.

Tolerances, written before the first run.  A rounding to a type is off by at most half a
step, h(T) = finfo(T).eps / 2 of the value.  With p the exact weights, A = sum_j p_j |v_j|
and n the keys of a row:
  * the output's own rounding: h(out) |o|;
  * weights rounded to a 16-bit type W: h(W) A, and n * 2^-25 * max|v| where W is fp16
    (half its smallest step; the largest unnormalised weight is at least 1);
  * cached values rounded to fp16: h(fp16) A;
  * an error e of an exponent z multiplies a weight by 1 + e, and so do the others' through
    the sum: 2 e A.  Products are exact in fp32; a sum of terms that is accumulated in fp32
    (tensor cores may cut instead of round: a whole step, 2^-23 of the largest partial sum,
    for each of the D / 16 steps) gives e <= scale * D/16 * 2^-23 * sum |terms|, where the
    cache's terms are |q_c| (base + 15) d with base 64 (fp16) or 128 (bf16);
  * exp2, the sums and the division in fp32: 2^-18 A covers them for n <= 2^17 positive
    terms summed in 8 or more parallel chains of rounding errors below 2^-24 each.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def moe():
    import expert_cache_host_router_b200 as m
    return m


def half(t):
    return torch.finfo(t).eps / 2


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def rnd(*shape, dtype=F32, seed=0, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(*shape, device=DEV, generator=g) * std).to(dtype)


def starts(lens):
    return [0] + np.cumsum(lens).tolist()


def quantised(x):
    """What the cache holds for x [..., D], in 64 bits (16-bit and plain fp32 inputs)."""
    b = x.double().unflatten(-1, (-1, 32))
    big = b.abs().amax(-1, keepdim=True)
    m = b.gather(-1, (b.abs() == big).to(torch.int8).argmax(-1, keepdim=True))
    d = (-m / 8).clamp(-8188, 8188)
    q = torch.where(d == 0, torch.full_like(b, 8.0), torch.floor(b / d + 8.5)).clamp(0, 15)
    return ((q - 8) * d.half().double()).flatten(-2)


def tables(seqs, width, first=0, seed=0):
    p = torch.randperm(seqs * width, generator=torch.Generator().manual_seed(seed)) + first
    return p.to(torch.int32).view(seqs, width).to(DEV)


class Cache:
    """A filled cache and, per sequence, the values it stands for [len, heads, D] in 64 bits."""

    def __init__(self, moe, lens, heads, dim, page, dtype=BF, seed=0, more=0, width=None, std=1.0):
        width = max(1, -(-max(lens) // page)) if width is None else width
        self.pool = moe.kv_pool(len(lens) * width + more, page, heads, dim)
        self.pool.fill_(0xFF)  # rows that nothing wrote: NaN scales
        self.table = tables(len(lens), width, seed=seed)
        self.lens = ints(lens)
        n = sum(lens)
        k, v = rnd(n, heads, dim, dtype=dtype, seed=seed + 1, std=std), rnd(n, heads, dim, dtype=dtype, seed=seed + 2, std=std)
        moe.kv_store(self.pool, k, v, self.table, ints(starts(lens)))
        cu = starts(lens)
        self.k = [quantised(k[a:b]) for a, b in zip(cu, cu[1:])]
        self.v = [quantised(v[a:b]) for a, b in zip(cu, cu[1:])]


def reference(q, k, v, scale):
    """o, A, z's, p of q [hq, D] over k, v [n, heads, D], all in 64 bits."""
    g = q.shape[0] // k.shape[1]
    z = torch.einsum("hgd,nhd->hgn", q.double().unflatten(0, (-1, g)), k) * scale
    p = torch.softmax(z, -1)
    return torch.einsum("hgn,nhd->hgd", p, v).flatten(0, 1), torch.einsum("hgn,nhd->hgd", p, v.abs()).flatten(0, 1), p


def z_error(q, k, scale):
    base = 64 if q.dtype == FP else 128
    d = (k.abs().unflatten(-1, (-1, 32)).amax(-1) / 7).amax()  # at least the largest scale
    return float(scale * q.shape[-1] / 16 * 2.0 ** -23 * (base + 15) * d * q.double().abs().sum(-1).max())


def check_attend(out, score_add, q, c, b, scale):
    n = c.k[b].shape[0]
    if n == 0:
        assert torch.equal(out[b], torch.zeros_like(out[b]))
        return
    o, A, p = reference(q[b], c.k[b], c.v[b], scale)
    e = 2 * z_error(q, c.k[b], scale) + 2.0 ** -18
    tol = half(q.dtype) * o.abs() + A * (2 * half(FP) + e) * (1 + half(q.dtype)) + n * 2.0 ** -25 * c.v[b].abs().max() + 2.0 ** -24
    err = (out[b].double() - o).abs()
    assert bool((err <= tol).all()), (b, n, float((err / tol).max()))
    if score_add is not None:
        w = p.sum(1)
        assert bool(((score_add[b, :, :n] - w).abs() <= w * e + 2.0 ** -22).all())


# ------------------------------------------------------------------ store and load


@pytest.mark.parametrize("dtype", [BF, FP, F32])
@pytest.mark.parametrize("dim,heads,page", [(64, 1, 16), (64, 3, 48), (128, 2, 64), (128, 5, 16)])
def test_store_then_load_is_the_definition(moe, dtype, dim, heads, page):
    lens, start = [1, 0, 70, 17, 33], [5, 3, 0, 15, 31]
    n = sum(lens)
    k, v = rnd(n, heads, dim, dtype=dtype, seed=3), rnd(n, heads, dim, dtype=dtype, seed=4, std=1e-3)
    table = tables(5, -(-110 // page))
    pool = moe.kv_pool(table.numel(), page, heads, dim)
    cu, st = ints(starts(lens)), ints(start)
    err = ints([0])
    moe.kv_store(pool, k, v, table, cu, st, error=err)
    gk, gv = moe.kv_load(pool, table, cu, st, n, F32, error=err)
    # fp32 sources: x / d in fp32 may round over a border that 64 bits do not cross, by one step d
    for got, x in ((gk, k), (gv, v)):
        ref = quantised(x)
        if dtype == F32:
            d = x.double().unflatten(-1, (-1, 32)).abs().amax(-1, keepdim=True) / 8
            off = (got.double() - ref).abs().unflatten(-1, (-1, 32))
            assert bool((off <= d * 1.001).all()) and float((off > 0).float().mean()) < 1e-4
        else:
            assert torch.equal(got.double(), ref)
    assert int(err) == 0
    for t in (BF, FP):
        hk, hv = moe.kv_load(pool, table, cu, st, n, t)
        assert torch.equal(hk, gk.to(t)) and torch.equal(hv, gv.to(t))


def test_store_touches_only_its_rows(moe):
    """Single tokens into every place of a tile, one after the other, give the bytes of one call."""
    dim, heads, page = 64, 2, 32
    k, v = rnd(40, heads, dim, dtype=BF, seed=1), rnd(40, heads, dim, dtype=BF, seed=2)
    table = tables(1, 2)
    one, many = moe.kv_pool(2, page, heads, dim), moe.kv_pool(2, page, heads, dim)
    one.fill_(0xA5), many.fill_(0xA5)
    moe.kv_store(one, k, v, table, ints([0, 40]))
    for i in torch.randperm(40, generator=torch.Generator().manual_seed(0)).tolist():
        moe.kv_store(many, k[i:i + 1], v[i:i + 1], table, ints([0, 1]), ints([i]))
    assert torch.equal(one, many)
    assert int((one == 0xA5).sum()) > 24 * heads * dim  # rows 40..63 are as they were


@pytest.mark.parametrize("how", ["heads outside", "odd offset", "expanded"])
def test_strides(moe, how):
    n, heads, dim = 21, 3, 64
    if how == "heads outside":
        k, v = (rnd(heads, n, dim, dtype=BF, seed=s).transpose(0, 1) for s in (1, 2))
    elif how == "odd offset":
        k, v = (rnd(n * heads * (dim + 3) + 1, dtype=BF, seed=s)[1:].view(n, heads, dim + 3)[..., :dim] for s in (1, 2))
    else:
        k, v = (rnd(n, 1, dim, dtype=BF, seed=s).expand(n, heads, dim) for s in (1, 2))
    table = tables(1, 2)
    pool = moe.kv_pool(2, 16, heads, dim)
    cu = ints([0, n])
    moe.kv_store(pool, k, v, table, cu)
    gk, gv = moe.kv_load(pool, table, cu, None, n, F32)
    assert torch.equal(gk.double(), quantised(k)) and torch.equal(gv.double(), quantised(v))
    out = tuple(torch.full((heads, n, dim + 1), 7.0, device=DEV)[..., :dim].transpose(0, 1) for _ in range(2))
    moe.kv_load(pool, table, cu, None, n, F32, out=out)
    assert torch.equal(out[0], gk) and torch.equal(out[1], gv)


def test_special_values(moe):
    x = torch.zeros(1, 1, 128, device=DEV)
    x[0, 0, :32] = 0.0
    x[0, 0, 32:64] = torch.linspace(-3, 3, 32)  # a tie of magnitudes: the first (negative) one decides
    x[0, 0, 64:96] = 1.0
    x[0, 0, 70] = float("nan")
    x[0, 0, 96] = float("inf")
    x[0, 0, 97] = -2e5
    table, cu = tables(1, 1), ints([0, 1])
    pool = moe.kv_pool(1, 16, 1, 128)
    moe.kv_store(pool, x, x, table, cu)
    for got in moe.kv_load(pool, table, cu, None, 1, F32):
        got = got[0, 0]
        assert torch.equal(got[:32], torch.zeros(32, device=DEV))
        assert torch.equal(got[32:64].double(), quantised(x)[0, 0, 32:64])
        assert bool(got[64:96].isnan().all())
        assert got[96] == 65504.0 and got[97] == -7 * 8188.0 or got[97] == -8 * 8188.0 + 8188.0


def test_padding_and_bad_places(moe):
    heads, dim = 2, 64
    k, v = rnd(12, heads, dim, dtype=FP, seed=1), rnd(12, heads, dim, dtype=FP, seed=2)
    table = ints([[0, 1], [99, 2], [-1, 3]])
    pool = moe.kv_pool(4, 16, heads, dim)
    pool.fill_(0x5A)
    err = ints([0])
    # rows 0 and 11 are padding; sequence 1's first page and sequence 2's first page do not exist
    cu, start = ints([1, 4, 8, 11]), ints([0, 14, 31])
    moe.kv_store(pool, k, v, table, cu, start, error=err)
    assert int(err) == moe.MOE_DEVERR_PAGE
    out = tuple(torch.full((12, heads, dim), 3.0, device=DEV) for _ in range(2))
    err.zero_()
    moe.kv_load(pool, table, cu, start, 12, F32, out=out, error=err)
    assert int(err) == moe.MOE_DEVERR_PAGE
    for got, x in zip(out, (k, v)):
        ref = quantised(x)
        for i in (1, 2, 3, 6, 7, 8):  # sequence 1: positions 14, 15 are on the missing page; sequence 2: 31 is the last
            assert torch.equal(got[i].double(), ref[i]), i
        for i in (4, 5, 9, 10):
            assert bool(got[i].isnan().all()), i
        for i in (0, 11):
            assert bool((got[i] == 3.0).all())
    moe.kv_store(pool, k, v, table, cu, ints([-5, 0, 2 ** 31 - 1]), error=err)  # positions below 0 and past the table
    assert int(err) == moe.MOE_DEVERR_PAGE


# ------------------------------------------------------------------ attend

LENS = [1, 0, 15, 16, 17, 33, 300, 2, 1029]


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim,heads,group,page", [(128, 2, 8, 64), (128, 1, 1, 16), (64, 3, 5, 48), (64, 2, 16, 16),
                                                  (128, 2, 12, 32), (64, 1, 40, 128), (128, 1, 17, 16)])
@pytest.mark.parametrize("scored", [False, True])
def test_attend(moe, dtype, dim, heads, group, page, scored):
    c = Cache(moe, LENS, heads, dim, page, dtype)
    q = rnd(len(LENS), heads * group, dim, dtype=dtype, seed=9, std=2.0)
    s0 = torch.rand(len(LENS), heads, 1100, device=DEV)
    score = s0.clone() if scored else None
    err = ints([0])
    out = moe.kv_attend(c.pool, q, c.table, c.lens, 1029, score=score, error=err)
    assert int(err) == 0
    add = None if score is None else score.double() - s0.double()
    for b, n in enumerate(LENS):
        check_attend(out, add, q, c, b, dim ** -0.5)
        if scored:
            assert torch.equal(score[b, :, n:], s0[b, :, n:])
    again = moe.kv_attend(c.pool, q, c.table, c.lens, 1029)
    assert torch.equal(out, again)  # with and without scores, run to run


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("n", [4097, 70001])
def test_attend_long(moe, dtype, n):
    """One sequence over many CTAs, weights that peak late so that running maxima move."""
    c = Cache(moe, [n], 2, 128, 64, dtype, std=2.0)
    q = rnd(1, 16, 128, dtype=dtype, seed=5, std=3.0)
    score = torch.zeros(1, 2, n, device=DEV)
    out = moe.kv_attend(c.pool, q, c.table, c.lens, n, score=score)
    check_attend(out, score.double(), q, c, 0, 128 ** -0.5)
    assert abs(float(score.double().sum()) - 16) < 16 * 2.0 ** -12


@pytest.mark.parametrize("scale", [1e-6, 0.5, 3.0])
def test_attend_scale(moe, scale):
    c = Cache(moe, [200, 40], 2, 64, 32, FP)
    q = rnd(2, 8, 64, dtype=FP, seed=5)
    out = moe.kv_attend(c.pool, q, c.table, c.lens, scale=scale)
    for b in range(2):
        check_attend(out, None, q, c, b, scale)


def test_attend_many_short_sequences(moe):
    """More sequences than CTAs, segments that start and end inside every run."""
    lens = [(7 * i) % 61 for i in range(1500)]
    c = Cache(moe, lens, 2, 64, 16, BF)
    q = rnd(1500, 8, 64, dtype=BF, seed=5)
    out = moe.kv_attend(c.pool, q, c.table, c.lens, 61)
    for b in list(range(0, 1500, 97)) + [1499]:
        check_attend(out, None, q, c, b, 64 ** -0.5)
    assert bool(out.isfinite().all())


@pytest.mark.parametrize("dim,heads,group", [(64, 2, 4), (128, 1, 40), (64, 3, 12)])
def test_attend_one_long_sequence_among_short_ones(moe, dim, heads, group):
    """Items of one piece and of very many in one call; scores of far fewer keys than max_len allows."""
    lens = [(5 * i) % 40 for i in range(47)] + [30000] + [17] * 16
    c = Cache(moe, lens, heads, dim, 64, BF)
    q = rnd(len(lens), heads * group, dim, dtype=BF, seed=5, std=2.0)
    s0 = torch.rand(len(lens), heads, 30000, device=DEV)
    score = s0.clone()
    out = moe.kv_attend(c.pool, q, c.table, c.lens, 30000, score=score)
    for b in (0, 1, 7, 46, 47, 48, len(lens) - 1):
        check_attend(out, score.double() - s0.double(), q, c, b, dim ** -0.5)
        assert torch.equal(score[b, :, lens[b]:], s0[b, :, lens[b]:])
    assert torch.equal(out, moe.kv_attend(c.pool, q, c.table, c.lens, 30000))


def test_attend_strides_and_out(moe):
    c = Cache(moe, [50, 61], 2, 128, 16, BF)
    q = rnd(8, 2, 131, dtype=BF, seed=5)[..., 1:129].transpose(0, 1)  # heads outside, odd offset
    out = torch.full((8, 2, 130), 5.0, dtype=BF, device=DEV)
    got = moe.kv_attend(c.pool, q, c.table, c.lens, out=out[..., 1:129].transpose(0, 1))
    ref = moe.kv_attend(c.pool, q.contiguous(), c.table, c.lens)
    assert torch.equal(got, ref)
    assert bool((out[..., 0] == 5).all()) and bool((out[..., 129] == 5).all())
    wide = torch.full((4, c.table.shape[1] + 3), -7, dtype=torch.int32, device=DEV)
    wide[1:3, 1:-2] = c.table
    assert torch.equal(moe.kv_attend(c.pool, q, wide[1:3, 1:-2], c.lens), ref)
    assert torch.equal(moe.kv_attend(c.pool, q, c.table[:, :], c.lens, max_len=10 ** 4), ref)


def test_attend_bad_sequences_are_nan_alone(moe):
    lens = [100, 40, 64, 20, 30]
    c = Cache(moe, lens, 2, 64, 16, FP)
    q = rnd(5, 4, 64, dtype=FP, seed=5)
    table, bad = c.table.clone(), c.lens.clone()
    table[0, 3] = c.pool.shape[0]       # a page that is not there
    table[4, 5] = -9                    # behind the end: not looked at
    bad[1], bad[3] = 101, -1            # past max_len, negative
    err = ints([0])
    out = moe.kv_attend(c.pool, q, table, bad, 100, error=err)
    assert int(err) == moe.MOE_DEVERR_PAGE
    for b in (0, 1, 3):
        assert bool(out[b].isnan().all())
    # not compared bit for bit with a good batch: the work is cut along all lengths, so where a
    # sequence's sum is split depends on the others (the tolerance above covers any split)
    for b in (2, 4):
        check_attend(out, None, q, c, b, 64 ** -0.5)


def test_attend_shared_pages_and_non_finite_neighbours(moe):
    """Two sequences share their first page; rows behind the ends are NaN (0xFF bytes)."""
    c = Cache(moe, [64, 64], 1, 64, 64, BF)
    table = torch.stack([c.table[0], c.table[0]])
    q = rnd(2, 4, 64, dtype=BF, seed=5)
    out = moe.kv_attend(c.pool, q, table, ints([64, 21]), 64)
    c.k, c.v = [c.k[0], c.k[0][:21]], [c.v[0], c.v[0][:21]]
    for b in range(2):
        check_attend(out, None, q, c, b, 64 ** -0.5)


def test_pool_past_32_bits(moe):
    pages, page, heads, dim = 500000, 64, 1, 128  # 4.6 GB
    pool = moe.kv_pool(pages, page, heads, dim)
    assert pool.numel() > 2 ** 32
    table = ints([[499999, 2, 499998]])
    n = 150
    k, v = rnd(n, heads, dim, dtype=BF, seed=1), rnd(n, heads, dim, dtype=BF, seed=2)
    cu = ints([0, n])
    moe.kv_store(pool, k, v, table, cu)
    gk, gv = moe.kv_load(pool, table, cu, None, n, F32)
    assert torch.equal(gk.double(), quantised(k)) and torch.equal(gv.double(), quantised(v))
    q = rnd(1, 8, dim, dtype=BF, seed=3)
    small = moe.kv_pool(3, page, heads, dim)
    moe.kv_store(small, k, v, ints([[0, 1, 2]]), cu)
    assert torch.equal(moe.kv_attend(pool, q, table, ints([n])), moe.kv_attend(small, q, ints([[0, 1, 2]]), ints([n])))


def test_streams_and_graphs(moe):
    """Calls on a stream of their own and replayed graphs (each with its own workspace, lengths
    and rows changed between replays) give what eager calls give."""
    c = Cache(moe, [300, 77], 2, 128, 64, BF, width=6)
    q = rnd(2, 16, 128, dtype=BF, seed=5)
    ref = moe.kv_attend(c.pool, q, c.table, c.lens)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = moe.kv_attend(c.pool, q, c.table, c.lens, stream=side)
    side.synchronize()
    assert torch.equal(out, ref)
    lens, qs = c.lens.clone(), q.clone()
    score = torch.zeros(2, 2, 384, device=DEV)
    graphs = []
    torch.cuda.synchronize()
    for scored in (False, True):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = moe.kv_attend(c.pool, qs, c.table, lens, 384, score=score if scored else None)
        graphs.append((g, o))
    for step in range(3):
        lens.copy_(c.lens - 5 * step)
        qs.copy_(q * (1 + step))
        score.zero_()
        for g, _ in graphs:
            g.replay()
        torch.cuda.synchronize()
        s = torch.zeros_like(score)
        want = moe.kv_attend(c.pool, qs, c.table, lens, 384, score=s)
        assert all(torch.equal(o, want) for _, o in graphs)
        assert torch.equal(s, score)


def test_two_streams_at_once(moe):
    """Different batches on two streams, interleaved many times without waiting in between."""
    a, b = (Cache(moe, lens, 2, 128, 64, BF, seed=s) for lens, s in (([900, 33, 4000], 1), ([2500, 7], 2)))
    qa, qb = rnd(3, 16, 128, dtype=BF, seed=5), rnd(2, 16, 128, dtype=BF, seed=6)
    ra, rb = moe.kv_attend(a.pool, qa, a.table, a.lens), moe.kv_attend(b.pool, qb, b.table, b.lens)
    pa = moe.attend_prompt(qa.repeat(100, 1, 1), qa[:, :2].repeat(100, 1, 1), qa[:, 2:4].repeat(100, 1, 1), ints([0, 300]))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        outs.append((moe.kv_attend(a.pool, qa, a.table, a.lens, stream=s1), ra))
        outs.append((moe.kv_attend(b.pool, qb, b.table, b.lens, stream=s2), rb))
        with torch.cuda.stream(s2):
            q3 = qa.repeat(100, 1, 1)
            outs.append((moe.attend_prompt(q3, q3[:, :2], q3[:, 2:4], ints([0, 300])), pa))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in outs)


def test_first_calls_of_a_process_can_be_captured(moe):
    """Every operator captured before it ever ran in the process, then replayed twice."""
    import subprocess
    import sys
    code = """
import torch, expert_cache_host_router_b200 as moe
d = "cuda:0"
i = lambda v: torch.tensor(v, dtype=torch.int32, device=d)
pool = moe.kv_pool(8, 16, 2, 64)
q = torch.randn(40, 4, 64, device=d).half(); k = torch.randn(40, 2, 64, device=d).half(); v = torch.randn(40, 2, 64, device=d).half()
table, out_table, cu, cu20, lens, score = i([[0, 1, 2]]), i([[3, 4]]), i([0, 40]), i([0, 20]), i([40]), torch.zeros(1, 2, 48, device=d)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    p = moe.attend_prompt(q, k, v, cu)
    moe.kv_store(pool, k, v, table, cu)
    o = moe.kv_attend(pool, q[39:], table, lens, 48, score=score)
    n, kept, s = moe.kv_evict(pool, table, lens, 48, score, 20, 4, out_table)
    kk, vv = moe.kv_load(pool, out_table, cu20, None, 20, torch.float16)
score.zero_()
g.replay(); torch.cuda.synchronize()
first = [x.clone() for x in (p, o, kept, s)]
score.zero_()
g.replay(); torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(first, (p, o, kept, s)))
assert torch.equal(p, moe.attend_prompt(q, k, v, cu)) and torch.equal(o, moe.kv_attend(pool, q[39:], table, lens, 48))
assert int(n) == 20 and kept[0, 0, -4:].tolist() == [36, 37, 38, 39]
print("captured")
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=200)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_own_workspace(moe):
    c = Cache(moe, [100, 4000], 2, 64, 32, FP)
    q = rnd(2, 8, 64, dtype=FP, seed=5)
    need = moe.kv_attend_workspace(c.pool, c.table, 8, 4000)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=DEV)
    ref = moe.kv_attend(c.pool, q, c.table, c.lens, 4000)
    assert torch.equal(moe.kv_attend(c.pool, q, c.table, c.lens, 4000, workspace=ws), ref)
    assert torch.equal(moe.kv_attend(c.pool, q, c.table, c.lens, 4000, workspace=ws), ref)
    with pytest.raises(moe.MoEError):
        moe.kv_attend(c.pool, q, c.table, c.lens, 4000, workspace=ws[:need - 256])
    assert moe.kv_attend_workspace(c.pool, c.table, 8, 4000, True) > need


@pytest.mark.parametrize("scale", [1e-30, 1.0, 1e30])
def test_attend_query_range(moe, scale):
    """Queries far from 1 in size: scaled to the fp16 range by powers of two inside."""
    c = Cache(moe, [70], 1, 64, 16, BF)
    q = rnd(1, 4, 64, dtype=F32, seed=5).mul(scale).to(BF)
    out = moe.kv_attend(c.pool, q, c.table, c.lens, scale=0.2 / scale if scale > 1e-20 else 0.2)
    o, A, _ = reference(q[0].double(), c.k[0], c.v[0], 0.2 / scale if scale > 1e-20 else 0.2)
    assert float((out[0].double() - o).abs().max()) <= 2.0 ** -7 * float(A.max())


@pytest.mark.parametrize("bad", ["table dtype", "lens count", "q head dim", "q rows", "q dtype", "score small", "score dtype",
                                 "pool view", "out shape", "lens float", "cu count", "mixed types", "evict same table", "keep 0"])
def test_binding_refusals_on_the_gpu(moe, bad):
    c = Cache(moe, [30, 40], 2, 64, 16, FP, more=8)
    q, k = rnd(2, 4, 64, dtype=FP), rnd(5, 2, 64, dtype=FP)
    cu, score = ints([0, 2, 5]), torch.zeros(2, 2, 48, device=DEV)
    call = {
        "table dtype": lambda: moe.kv_attend(c.pool, q, c.table.long(), c.lens),
        "lens count": lambda: moe.kv_attend(c.pool, q, c.table, c.lens[:1]),
        "lens float": lambda: moe.kv_attend(c.pool, q, c.table, c.lens.float()),
        "q head dim": lambda: moe.kv_attend(c.pool, rnd(2, 4, 128, dtype=FP), c.table, c.lens),
        "q rows": lambda: moe.kv_attend(c.pool, q[:1], c.table, c.lens),
        "q dtype": lambda: moe.kv_attend(c.pool, q.float(), c.table, c.lens),
        "score small": lambda: moe.kv_attend(c.pool, q, c.table, c.lens, 48, score=score[..., :40]),
        "score dtype": lambda: moe.kv_attend(c.pool, q, c.table, c.lens, 48, score=score.double()),
        "pool view": lambda: moe.kv_attend(c.pool[:, :1], q, c.table, c.lens),
        "out shape": lambda: moe.kv_attend(c.pool, q, c.table, c.lens, out=q[:, :2]),
        "cu count": lambda: moe.kv_store(c.pool, k, k, c.table, cu[:2]),
        "mixed types": lambda: moe.kv_store(c.pool, k, k.float(), c.table, cu),
        "evict same table": lambda: moe.kv_evict(c.pool, c.table, c.lens, 48, score, 16, 4, c.table),
        "keep 0": lambda: moe.kv_evict(c.pool, c.table, c.lens, 48, score, 0, 0, ints([[6], [7]])),
    }[bad]
    with pytest.raises(moe.MoEError) as e:
        call()
    assert e.value.status == moe.MOE_ERR_INVALID


# ------------------------------------------------------------------ evict


def evict_reference(score, n, keep, recent):
    s = score[:n].clone()
    s[s.isnan()] = -float("inf")
    if n <= keep:
        return list(range(n))
    old = sorted(range(n - recent), key=lambda i: (-float(s[i]), bool(score[i].isnan()), i))[: keep - recent]
    return sorted(old) + list(range(n - recent, n))


@pytest.mark.parametrize("dim,heads,page", [(128, 2, 64), (64, 3, 16), (64, 1, 48)])
@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (37, 5), (64, 64), (100, 0), (255, 31)])
def test_evict(moe, dim, heads, page, keep, recent):
    lens = [0, 1, 36, 37, 38, 101, 256, 700]
    width = -(-keep // page)
    c = Cache(moe, lens, heads, dim, page, FP, more=len(lens) * width)
    g = torch.Generator(device=DEV).manual_seed(2)
    score = torch.randint(0, 12, (len(lens), heads, 700), device=DEV, generator=g).float() / 4  # many ties
    score[5, 0, ::3] = float("nan")
    score[6, :, 10:20] = -0.0
    score[6, :, 20:30] = -1.5
    score[7, 0, 5] = float("inf")
    out_table = tables(len(lens), width, first=c.table.numel())
    before = c.pool.clone()
    out_lens, kept, out_score = moe.kv_evict(c.pool, c.table, c.lens, 700, score, keep, recent, out_table)
    old = c.table.flatten().long()
    assert torch.equal(c.pool[old], before[old])
    rows, ks, vs = [], [], []
    cpu = score.cpu()
    for b, n in enumerate(lens):
        assert int(out_lens[b]) == min(n, keep)
        for h in range(heads):
            ref = evict_reference(cpu[b, h], n, keep, recent)
            m = len(ref)
            assert kept[b, h].tolist() == ref + [-1] * (keep - m), (b, h)
            want = torch.zeros(keep, device=DEV)
            want[:m] = score[b, h, ref]
            assert torch.equal(out_score[b, h].nan_to_num(-9), want.nan_to_num(-9))
    cu = ints(starts([min(n, keep) for n in lens]))
    gk, gv = moe.kv_load(c.pool, out_table, cu, None, int(cu[-1]), F32)
    at = 0
    for b, n in enumerate(lens):
        m = min(n, keep)
        for h in range(heads):
            idx = kept[b, h, :m].long()
            assert torch.equal(gk[at:at + m, h].double(), c.k[b][idx, h]) and torch.equal(gv[at:at + m, h].double(), c.v[b][idx, h])
        # rows behind the new length are left as they were
        tile, r = m // 16, m % 16
        if m < keep and r:
            page_id = int(out_table[b, m // page])
            got, was = c.pool[page_id, 0, tile % (page // 16)], before[page_id, 0, tile % (page // 16)]
            row = 16 * (dim // 32)
            assert torch.equal(got[r * row:16 * row], was[r * row:16 * row])
            assert torch.equal(got[16 * dim + r * (dim // 16):17 * dim], was[16 * dim + r * (dim // 16):17 * dim])
            vp = got[8 * dim:16 * dim].view(8, dim // 4, 2, 2), was[8 * dim:16 * dim].view(8, dim // 4, 2, 2)
            for i in range(r, 16):
                assert torch.equal(vp[0][i // 2, :, i % 2], vp[1][i // 2, :, i % 2])
        at += m


def test_evict_large_scores_and_bad_lengths(moe):
    n, keep = 40000, 9001
    c = Cache(moe, [n, 50], 1, 64, 64, BF, more=2 * 141)
    score = torch.rand(2, 1, n, device=DEV) ** 16  # most of them in a few binades
    err = ints([0])
    lens = c.lens.clone()
    lens[1] = n + 1
    out_table = tables(2, 141, first=c.table.numel())
    out_lens, kept, _ = moe.kv_evict(c.pool, c.table, lens, n, score, keep, 100, out_table, error=err)
    assert out_lens.tolist() == [keep, 0] and int(err) == moe.MOE_DEVERR_PAGE
    assert kept[0, 0].tolist() == evict_reference(score[0, 0].cpu(), n, keep, 100)
    assert bool((kept[1] == -1).all())


# ------------------------------------------------------------------ prompts


def check_prompt(out, q, k, v, cu, scale):
    g = q.shape[1] // k.shape[1]
    for a, b in zip(cu, cu[1:]):
        for h in range(q.shape[1]):
            qq, kk, vv = q[a:b, h].double(), k[a:b, h // g].double(), v[a:b, h // g].double()
            n = b - a
            mask = torch.triu(torch.ones(n, n, dtype=torch.bool, device=DEV), 1)
            p = torch.softmax((qq @ kk.T * scale).masked_fill(mask, -math.inf), -1)
            o, A = p @ vv, p @ vv.abs()
            e = 2 * scale * q.shape[2] / 16 * 2.0 ** -23 * float((qq.abs() @ kk.abs().T).max()) if n else 0.0
            tol = half(q.dtype) * o.abs() + A * (half(q.dtype) + e + 2.0 ** -18) * (1 + half(q.dtype))
            if q.dtype == FP and n:
                tol = tol + n * 2.0 ** -25 * vv.abs().max()
            err = (out[a:b, h].double() - o).abs()
            assert bool((err <= tol + 2.0 ** -24).all()), (a, b, h, float((err / tol).max()))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim,hq,hkv", [(64, 4, 2), (128, 3, 1), (128, 2, 2)])
@pytest.mark.parametrize("lens", [[1], [2], [127], [128], [129], [255], [256], [257], [700], [1, 1, 130, 0, 513, 64, 3]])
def test_prompt(moe, dtype, dim, hq, hkv, lens):
    n = sum(lens)
    q = rnd(n, hq, dim, dtype=dtype, seed=1, std=2.0)
    k, v = rnd(n, hkv, dim, dtype=dtype, seed=2), rnd(n, hkv, dim, dtype=dtype, seed=3)
    cu = starts(lens)
    out = moe.attend_prompt(q, k, v, ints(cu))
    check_prompt(out, q, k, v, cu, dim ** -0.5)
    assert torch.equal(out, moe.attend_prompt(q, k, v, ints(cu)))


@pytest.mark.parametrize("dtype", [BF, FP])
def test_prompt_long_and_peaked(moe, dtype):
    """Running maxima that move in many tiles (large logits), 3001 tokens."""
    n = 3001
    q, k = rnd(n, 2, 128, dtype=dtype, seed=1, std=4.0), rnd(n, 1, 128, dtype=dtype, seed=2, std=2.0)
    v = rnd(n, 1, 128, dtype=dtype, seed=3)
    ramp = torch.linspace(0.5, 4, n, device=DEV)[:, None, None]
    k = (k.float() * ramp).to(dtype)
    out = moe.attend_prompt(q, k, v, ints([0, n]))
    check_prompt(out, q, k, v, [0, n], 128 ** -0.5)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim,hq,hkv,lens", [(128, 4, 1, [2100]), (64, 6, 3, [1024]), (64, 7, 7, [5101]), (128, 8, 2, [4096]),
                                             (128, 2, 1, [100, 2900, 300]), (64, 3, 1, [1500, 900, 700]), (64, 4, 4, [513, 5000, 0, 600])])
def test_prompt_pairs(moe, dtype, dim, hq, hkv, lens):
    """Few long items: two CTAs share each (one or several items in turn), odd and even tile counts."""
    n = sum(lens)
    q = rnd(n, hq, dim, dtype=dtype, seed=1, std=2.0)
    k, v = rnd(n, hkv, dim, dtype=dtype, seed=2), rnd(n, hkv, dim, dtype=dtype, seed=3)
    out = moe.attend_prompt(q, k, v, ints(starts(lens)))
    check_prompt(out, q, k, v, starts(lens), dim ** -0.5)
    assert torch.equal(out, moe.attend_prompt(q, k, v, ints(starts(lens))))


def test_prompt_packed_views_padding_and_neighbours(moe):
    """q, k, v as views of one fused tensor; rows outside the sequences stay; NaN and infinity in
    a neighbouring sequence and in the padding reach nothing."""
    n, hq, hkv, dim = 400, 4, 2, 64
    fused = rnd(n, hq + 2 * hkv, dim, dtype=BF, seed=1)
    cu = [3, 140, 141, 300]
    clean = fused.clone()
    fused[300:], fused[:3], fused[140] = float("nan"), float("inf"), float("nan")
    q, k, v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    out = torch.full((n, hq, dim + 2), 9.0, dtype=BF, device=DEV)
    moe.attend_prompt(q, k, v, ints(cu), out=out[..., 1:dim + 1])
    c = clean[:, :hq], clean[:, hq:hq + hkv], clean[:, hq + hkv:]
    for a, b in ((3, 140), (141, 300)):
        check_prompt(out[..., 1:dim + 1], *c, [a, b], dim ** -0.5)
    assert bool(out[140, :, 1:dim + 1].isnan().all())
    assert bool((out[:3] == 9).all()) and bool((out[300:] == 9).all())
    assert bool((out[..., 0] == 9).all()) and bool((out[..., dim + 1] == 9).all())


def test_prompt_strides_without_meaning_and_of_zero(moe):
    """Strides of a single head or row are not looked at; heads that share one row are refused."""
    n, dim = 200, 64
    q, k, v = rnd(n, 4, dim, dtype=BF, seed=1), rnd(n, dim, dtype=BF, seed=2), rnd(n, dim, dtype=BF, seed=3)
    cu = ints([0, n])
    want = moe.attend_prompt(q, k[:, None], v[:, None], cu)
    check_prompt(want, q, k[:, None], v[:, None], [0, n], dim ** -0.5)
    odd = [x.as_strided((n, 1, dim), (dim, 1, 1)) for x in (k, v)]
    assert torch.equal(want, moe.attend_prompt(q, *odd, cu))
    row = [x[:1].as_strided((1, 4, dim), (3, dim, 1)) for x in (q, q, q)]
    assert torch.equal(moe.attend_prompt(*row, ints([0, 1])), q[:1])  # one key: its own value
    for bad in ((q, k[:, None].expand(n, 4, dim), v[:, None]), (q, k[:, None], v[:1, None].expand(n, 1, dim))):
        with pytest.raises(moe.MoEError):
            moe.attend_prompt(*bad, cu)
    with pytest.raises(moe.MoEError):
        moe.attend_prompt(q, k[:, None], v[:, None], cu, out=torch.empty_like(q[:, :1]).expand(n, 4, dim))


def test_prompt_bad_bounds(moe):
    n = 300
    q = rnd(n, 2, 64, dtype=FP, seed=1)
    err = ints([0])
    out = torch.full_like(q, 4.0)
    moe.attend_prompt(q, q, q, ints([0, 100, 90, 301]), out=out, error=err)
    assert int(err) == moe.MOE_DEVERR_PAGE
    check_prompt(out, q, q, q, [0, 100], 64 ** -0.5)
    assert bool((out[100:] == 4).all())


def test_prompt_many_sequences_and_graph(moe):
    lens = [(5 * i) % 23 for i in range(900)]
    n = sum(lens)
    q, k, v = rnd(n, 4, 64, dtype=BF, seed=1), rnd(n, 2, 64, dtype=BF, seed=2), rnd(n, 2, 64, dtype=BF, seed=3)
    cu = ints(starts(lens))
    out = moe.attend_prompt(q, k, v, cu)
    c = starts(lens)
    for b in range(0, 900, 83):
        check_prompt(out, q, k, v, c[b:b + 2], 64 ** -0.5)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        got = moe.attend_prompt(q, k, v, cu)
    for _ in range(2):
        q.copy_(torch.roll(q, 1, 0))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, moe.attend_prompt(q, k, v, cu))


# ------------------------------------------------------------------ together


def test_a_layer_served_together(moe):
    """Prompts, then decode steps over the 4-bit cache with weights summed, an eviction, and
    more steps, each checked against the rows that the cache stands for; the MoE step of
    the library runs on the attention output in between."""
    import synthetic
    from helpers import build_gpu, make_layers
    s = synthetic.Shape(n_layers=1, hidden=512, n_experts=64, top_k=4, inter=256, shared_inter=0, ring_slots=4, use_rmsnorm=1)
    layer = build_gpu(s, make_layers(s))
    layer.set_residency(1.0)
    lens, hq, hkv, dim, page = [37, 130], 4, 2, 128, 32
    n, keep, recent = sum(lens), 60, 16
    q, k, v = rnd(n, hq, dim, dtype=BF, seed=1), rnd(n, hkv, dim, dtype=BF, seed=2), rnd(n, hkv, dim, dtype=BF, seed=3)
    cu = starts(lens)
    out = moe.attend_prompt(q, k, v, ints(cu))
    check_prompt(out, q, k, v, cu, dim ** -0.5)
    y = layer.prefill(out.reshape(n, -1).float().contiguous())
    assert bool(y.isfinite().all())
    pool, table = moe.kv_pool(20, page, hkv, dim), tables(2, 6)
    moe.kv_store(pool, k, v, table, ints(cu))
    ks, vs = [quantised(k[a:b]) for a, b in zip(cu, cu[1:])], [quantised(v[a:b]) for a, b in zip(cu, cu[1:])]
    at, score = ints(lens), torch.zeros(2, hkv, 192, device=DEV)
    one = ints([0, 1, 2])
    exact = torch.zeros(2, hkv, 192, dtype=torch.float64, device=DEV)

    class View:
        pass

    for step in range(10):
        if step == 6:
            out_table = tables(2, 4, first=12)
            new, kept, score60 = moe.kv_evict(pool, table, at, 192, score, keep, recent, out_table)
            assert new.tolist() == [min(x, keep) for x in at.tolist()]
            for b in range(2):
                m = int(new[b])
                idx = kept[b, :, :m].long()
                ks[b] = torch.stack([ks[b][idx[h], h] for h in range(hkv)], 1)
                vs[b] = torch.stack([vs[b][idx[h], h] for h in range(hkv)], 1)
                ref = exact[b].gather(-1, idx)
                exact[b].zero_()
                exact[b, :, :m] = ref
            score.zero_()
            score[..., :keep] = score60
            table, at = out_table, new
        qs = rnd(2, hq, dim, dtype=BF, seed=50 + step)
        kn, vn = rnd(2, hkv, dim, dtype=BF, seed=70 + step), rnd(2, hkv, dim, dtype=BF, seed=90 + step)
        moe.kv_store(pool, kn, vn, table, one, at)
        at = at + 1
        o = moe.kv_attend(pool, qs, table, at, score=score)
        view = View()
        for b in range(2):
            ks[b], vs[b] = torch.cat([ks[b], quantised(kn[b:b + 1])]), torch.cat([vs[b], quantised(vn[b:b + 1])])
            _, _, p = reference(qs[b], ks[b], vs[b], dim ** -0.5)
            exact[b, :, :ks[b].shape[0]] += p.sum(1)
        view.k, view.v = ks, vs
        for b in range(2):
            check_attend(o, None, qs, view, b, dim ** -0.5)
            y = layer.decode(o[b].reshape(-1).float().contiguous())
            assert bool(y.isfinite().all())
    layer.sync()
    assert float((score.double() - exact).abs().max()) < 1e-4
    layer.close()
