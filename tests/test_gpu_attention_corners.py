"""Corners of the attention operators that tests/test_gpu_attention.py passes by.

Against 64 bits, with the tolerances that tests/test_gpu_attention.py derives."""
import math
import time

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_attention import BF, DEV, F32, FP, Cache, check_attend, half, ints, moe, quantised, rnd, starts, tables  # noqa: E402,F401
from prompt_items import turns  # noqa: E402
from test_prompt_items import SHORT_AMONG_LONG, SMS  # noqa: E402


def check_rows(out, q, k, v, first, n, rows, scale):
    """Rows `rows` (numbers within it) of the sequence first .. first + n - 1."""
    g = q.shape[1] // k.shape[1]
    at = torch.tensor(rows, device=DEV)
    for h in range(q.shape[1]):
        qq, kk, vv = q[first + at, h].double(), k[first:first + n, h // g].double(), v[first:first + n, h // g].double()
        later = torch.arange(n, device=DEV)[None, :] > at[:, None]
        p = torch.softmax((qq @ kk.T * scale).masked_fill(later, -math.inf), -1)
        o, A = p @ vv, p @ vv.abs()
        e = 2 * scale * q.shape[2] / 16 * 2.0 ** -23 * float((qq.abs() @ kk.abs().T).max())
        tol = half(q.dtype) * o.abs() + A * (half(q.dtype) + e + 2.0 ** -18) * (1 + half(q.dtype)) + 2.0 ** -24
        if q.dtype == FP:
            tol = tol + n * 2.0 ** -25 * vv.abs().max()
        err = (out[first + at, h].double() - o).abs()
        assert bool((err <= tol).all()), (first, h, float((err / tol).max()))


# ------------------------------------------------------------------ prompts


@pytest.mark.parametrize("dtype,dim", [(BF, 128), (FP, 64)])
@pytest.mark.parametrize("lens,heads", SHORT_AMONG_LONG)
def test_prompt_pairs_with_turns_without_key_tiles(moe, dtype, dim, lens, heads):
    assert torch.cuda.get_device_properties(0).multi_processor_count == SMS
    n = sum(lens)
    q = rnd(n, heads, dim, dtype=dtype, seed=1, std=2.0)
    k, v = rnd(n, 1, dim, dtype=dtype, seed=2), rnd(n, 1, dim, dtype=dtype, seed=3)
    err = ints([0])
    out = moe.attend_prompt(q, k, v, ints(starts(lens)), error=err)
    for _ in range(20):
        assert torch.equal(out, moe.attend_prompt(q, k, v, ints(starts(lens)), error=err))
    assert int(err) == 0
    for first, m in zip(starts(lens), lens):
        rows = sorted({i for i in [*range(min(m, 130)), *range(m // 2, m // 2 + 5), *range(m - 130, m)] if 0 <= i < m})
        check_rows(out, q, k, v, first, m, rows, dim ** -0.5)


# ------------------------------------------------------------------ attend: range of queries and scales


@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("power,scale", [(-80, 1e-30), (-80, 2.0 ** 76), (-80, 1e25), (-120, 2.0 ** 117), (-126, 1e-38), (0, 1e-45),
                                         (100, 2.0 ** -103), (126, 2.0 ** -126)])
def test_attend_queries_and_scales_far_from_one(moe, scored, power, scale):
    """Products of order 1 from tiny queries with a scale that makes up for it; equal weights where
    both are tiny; bf16 queries down to the subnormal ones."""
    c = Cache(moe, [70, 1, 600], 2, 64, 16, BF)
    q = rnd(3, 8, 64, seed=5).clamp(-1.9, 1.9).double().mul(2.0 ** power).to(BF)
    score = torch.zeros(3, 2, 600, device=DEV)
    out = moe.kv_attend(c.pool, q, c.table, c.lens, 600, scale=scale, score=score if scored else None)
    for b in range(3):
        check_attend(out, score.double() if scored else None, q, c, b, scale)


def test_attend_zero_queries_and_the_largest_scale(moe):
    c = Cache(moe, [70, 1], 1, 128, 16, FP)
    q = torch.zeros(2, 8, 128, dtype=FP, device=DEV)
    out = moe.kv_attend(c.pool, q, c.table, c.lens, scale=3.4e38)
    for b in range(2):
        check_attend(out, None, q, c, b, 1.0)


# ------------------------------------------------------------------ store: the bytes


def codes(pool, table, n, dim):
    """Codes and scales (keys, values) of the first n positions of one sequence and head 0, from the bytes."""
    nb = dim // 32
    raw = pool[table.long()][:, 0].reshape(-1, 18 * dim)
    kb = raw[:, :8 * dim].reshape(-1, 16, 4, nb, 4).transpose(2, 3).reshape(-1, nb, 16)
    vb = raw[:, 8 * dim:16 * dim].reshape(-1, 8, 8, nb, 2, 2).permute(0, 1, 4, 3, 2, 5).reshape(-1, nb, 16)
    kd = raw[:, 16 * dim:17 * dim].contiguous().view(FP).reshape(-1, nb)
    vd = raw[:, 17 * dim:].contiguous().view(FP).reshape(-1, 8, nb, 2).transpose(2, 3).reshape(-1, nb)
    return [(torch.cat([b & 15, b >> 4], -1)[:n].double(), d[:n]) for b, d in ((kb, kd), (vb, vd))]


@pytest.mark.parametrize("dtype,low,high", [(BF, -133, 127), (FP, -24, 15)])
def test_store_bytes_are_the_definition(moe, dtype, low, high):
    """Blocks of every magnitude that the type has, subnormal ones too, with zeros among their channels."""
    dim, reps = 64, 4
    power = torch.arange(low, high + 1, device=DEV).repeat_interleave(reps)
    n = power.numel()
    x = rnd(n, 2, dim, seed=3).clamp(-1.9, 1.9).double() * 2.0 ** power.double()[:, None, None]
    x[:, :, ::5] = 0
    x = x.clamp(-torch.finfo(dtype).max, torch.finfo(dtype).max).to(dtype)
    k, v = x[:, :1].contiguous(), x[:, 1:].contiguous()
    table = tables(1, -(-n // 16))
    pool = moe.kv_pool(table.numel(), 16, 1, dim)
    moe.kv_store(pool, k, v, table, ints([0, n]))
    for (q, d), rows in zip(codes(pool, table[0], n, dim), (k, v)):
        b = rows[:, 0].double().unflatten(-1, (-1, 32))
        big = b.abs().amax(-1, keepdim=True)
        m = b.gather(-1, (b.abs() == big).to(torch.int8).argmax(-1, keepdim=True))
        want_d = (-m / 8).clamp(-8188, 8188)
        want = torch.where(want_d == 0, torch.full_like(b, 8.0), torch.floor(b / want_d + 8.5)).clamp(0, 15)
        assert torch.equal(q, want)
        assert torch.equal(d.view(torch.int16), want_d.squeeze(-1).to(FP).view(torch.int16))


@pytest.mark.parametrize("dtype", [BF, FP, F32])
def test_store_special_values(moe, dtype):
    """Ties of magnitude (the first value decides), NaN (its whole block), infinities of both signs, zeros."""
    x = torch.zeros(5, 1, 64, dtype=dtype, device=DEV)
    x[0, 0, :32] = torch.linspace(-3, 3, 32).to(dtype)
    x[0, 0, 32:] = torch.linspace(3, -3, 32).to(dtype)
    x[1, 0, 3] = float("nan")
    x[2, 0, 7], x[2, 0, 8], x[2, 0, 9] = float("inf"), -float("inf"), 100.0
    x[3, 0, 7], x[3, 0, 8], x[3, 0, 9] = -float("inf"), float("inf"), -torch.finfo(FP).max
    x[4, 0, 40] = float("-nan")
    x[4, 0, 41] = float("inf")
    table, cu = tables(1, 1), ints([0, 5])
    pool = moe.kv_pool(1, 16, 1, 64)
    moe.kv_store(pool, x, x, table, cu)
    for got in moe.kv_load(pool, table, cu, None, 5, F32):
        got = got[:, 0]
        assert torch.equal(got[0].double(), quantised(x[0, 0]))
        assert got[0, 0] == -got[0, 32] and abs(float(got[0, 0])) == 3.0  # the deciding value is kept
        assert bool(got[1, :32].isnan().all()) and torch.equal(got[1, 32:], torch.zeros(32, device=DEV))
        assert float(got[2, 7]) == 65504.0 and float(got[2, 8]) == -7 * 8188.0 and float(got[2, 9]) == 0.0
        assert float(got[3, 7]) == -65504.0 and float(got[3, 8]) == 7 * 8188.0 and float(got[3, 9]) == -65504.0
        assert bool((got[2, 10:] == 0).all()) and bool((got[3, 10:] == 0).all())
        assert bool(got[4, 32:].isnan().all()) and bool((got[4, :32] == 0).all())


# ------------------------------------------------------------------ tables


def test_sequences_that_share_one_table_row(moe):
    """Several new tokens of one sequence, each a row of the batch: one table row for all of them."""
    n, t = 90, 5
    c = Cache(moe, [n], 2, 64, 16, FP)
    q = rnd(t, 4, 64, dtype=FP, seed=5)
    lens = ints([n - t + 1 + i for i in range(t)])
    shared = c.table.expand(t, -1)
    assert shared.stride(0) == 0
    score = torch.zeros(t, 2, n, device=DEV)
    out = moe.kv_attend(c.pool, q, shared, lens, n, score=score)
    assert torch.equal(out, moe.kv_attend(c.pool, q, shared.contiguous(), lens, n))
    c.k, c.v = ([x[0][:int(m)] for m in lens] for x in (c.k, c.v))
    for b in range(t):
        check_attend(out, score.double(), q, c, b, 64 ** -0.5)
    # their rows are written and read through it as well, each at a position of its own
    k, v = rnd(t, 2, 64, dtype=FP, seed=6), rnd(t, 2, 64, dtype=FP, seed=7)
    cu = ints(range(t + 1))
    moe.kv_store(c.pool, k, v, shared, cu, lens - 1)
    gk, gv = moe.kv_load(c.pool, shared, cu, lens - 1, t, F32)
    assert torch.equal(gk.double(), quantised(k)) and torch.equal(gv.double(), quantised(v))
    # cut down to different pages each
    more = moe.kv_pool(c.pool.shape[0] + t, 16, 2, 64)
    more[:c.pool.shape[0]] = c.pool
    new, kept, _ = moe.kv_evict(more, shared, lens, n, score, 16, 4, tables(t, 1, first=c.pool.shape[0]))
    assert new.tolist() == [16] * t and kept[0, 0, -4:].tolist() == [n - t - 3 + i for i in range(4)]
    with pytest.raises(moe.MoEError):  # but not to the same ones
        moe.kv_evict(more, shared, lens, n, score, 16, 4, tables(1, 1, first=c.pool.shape[0]).expand(t, -1))


# ------------------------------------------------------------------ gradients


@pytest.mark.parametrize("which", ["store", "attend", "prompt", "prompt values"])
def test_rows_that_want_a_gradient_are_refused(moe, which):
    """No gradient flows through these calls: a call that would lose one is refused, unless gradients are off."""
    c = Cache(moe, [40], 2, 64, 16, FP)
    q, k = rnd(1, 4, 64, dtype=FP).requires_grad_(), rnd(1, 2, 64, dtype=FP)
    call = {
        "store": lambda: moe.kv_store(c.pool, k, q[:, :2], c.table, ints([0, 1])),
        "attend": lambda: moe.kv_attend(c.pool, q, c.table, c.lens),
        "prompt": lambda: moe.attend_prompt(q, k, k, ints([0, 1])),
        "prompt values": lambda: moe.attend_prompt(q.detach(), k, q[:, :2], ints([0, 1])),
    }[which]
    with pytest.raises(moe.MoEError) as e:
        call()
    assert e.value.status == moe.MOE_ERR_UNSUPPORTED
    with torch.no_grad():
        call()
    with torch.inference_mode():
        call()


# ------------------------------------------------------------------ evict


@pytest.mark.parametrize("dim", [64, 128])
def test_evicted_rows_of_a_missing_page_are_nan(moe, dim):
    """Kept rows whose page is not there do not leave what was in their new place before."""
    n, keep = 80, 37
    c = Cache(moe, [n, n], 2, dim, 16, BF, more=6)
    score = torch.rand(2, 2, n, device=DEV)
    out_table = tables(2, 3, first=c.table.numel())
    moe.kv_store(c.pool, *(rnd(2 * 48, 2, dim, dtype=BF, seed=s) for s in (7, 8)), out_table, ints([0, 48, 96]))  # what was there before
    before = moe.kv_load(c.pool, out_table, ints([0, 48, 96]), None, 96, F32)
    table = c.table.clone()
    table[0, 2] = -1                # positions 32..47 of the first sequence
    err = ints([0])
    new, kept, _ = moe.kv_evict(c.pool, table, c.lens, n, score, keep, 5, out_table, error=err)
    assert int(err) == moe.MOE_DEVERR_PAGE and new.tolist() == [keep, keep]
    after = moe.kv_load(c.pool, out_table, ints([0, 48, 96]), None, 96, F32)
    for rows, got, was in ((c.k, *[x[0] for x in (after, before)]), (c.v, *[x[1] for x in (after, before)])):
        for b in range(2):
            for h in range(2):
                for r in range(48):
                    x = got[48 * b + r, h].double()
                    if r >= keep:
                        assert torch.equal(x, was[48 * b + r, h].double())
                    elif b == 0 and 32 <= int(kept[b, h, r]) < 48:
                        assert bool(x.isnan().all())
                    else:
                        assert torch.equal(x, rows[b][int(kept[b, h, r]), h])


# ------------------------------------------------------------------ errors


def test_a_refused_call_leaves_nothing_behind(moe):
    """A device that is not there: that call fails, the next good ones do not."""
    import ctypes
    P = ctypes.c_void_p
    c = Cache(moe, [40], 2, 64, 16, FP, more=4)
    k, cu, score = rnd(3, 2, 64, dtype=FP), ints([0, 3]), torch.zeros(1, 2, 48, device=DEV)
    out_table = tables(1, 1, first=c.table.numel())
    absent = moe.KvPool(c.pool.data_ptr(), c.pool.shape[0], 2, 64, 16, torch.cuda.device_count(), None)
    table = moe.KvTable(c.table.data_ptr(), 1, c.table.shape[1], c.table.shape[1])
    rows = moe.Rows(k.data_ptr(), k.stride(0), k.stride(1))

    def fail():
        L = moe.lib()
        s = L.moe_kv_store(absent, table, P(cu.data_ptr()), None, rows, rows, 3, moe.MOE_F16, None)
        a = L.moe_kv_attend_workspace(absent, table, 4, 40, 0, ctypes.c_size_t())
        p = L.moe_attend_prompt(torch.cuda.device_count(), rows, rows, rows, moe.Rows(score.data_ptr(), 128, 64), P(cu.data_ptr()), 1, 3,
                                2, 2, 64, moe.MOE_F16, 1.0, None, None)
        assert (s, a, p) == (moe.MOE_ERR_CUDA,) * 3
        with pytest.raises(moe.MoEError):
            moe.moe_create(moe.Config(1, 256, 16, 2, 256, 0, 0, 0, 1e-6, torch.cuda.device_count(), 0, 0))

    fail()
    moe.kv_store(c.pool, k, k, c.table, cu)
    fail()
    moe.kv_load(c.pool, c.table, cu, None, 3, FP)
    fail()
    moe.kv_evict(c.pool, c.table, c.lens, 48, score, 16, 4, out_table)
    fail()
    moe.kv_attend(c.pool, rnd(1, 4, 64, dtype=FP), c.table, c.lens)
    fail()
    moe.attend_prompt(k, k, k, cu)
    torch.cuda.synchronize()


# ------------------------------------------------------------------ prompts: what is not finite


def test_prompt_keys_that_no_row_can_see(moe):
    """A whole tile of keys with products of minus infinity has no weight; NaN in later keys reaches no earlier row."""
    n, dim = 520, 64
    q, k, v = rnd(n, 2, dim, dtype=BF, seed=1).abs(), rnd(n, 2, dim, dtype=BF, seed=2), rnd(n, 2, dim, dtype=BF, seed=3)
    k[:200, 0, 3] = -float("inf")
    k[400, 1] = float("nan")
    q[:, :, 3] = 1.0
    out = moe.attend_prompt(q, k, v, ints([0, n]))
    assert bool(out[:200, 0].isnan().all()) and bool(out[400:, 1].isnan().all())
    # without the rows of no weight
    shifted = out[200:, :1]
    check_rows(shifted, q[200:, :1], k[200:, :1], v[200:, :1], 0, n - 200, list(range(n - 200)), dim ** -0.5)
    check_rows(out[:, 1:], q[:, 1:], k[:, 1:], v[:, 1:], 0, 400, list(range(400)), dim ** -0.5)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim,hq,hkv,lens", [(64, 4, 2, [300]), (128, 2, 1, [129, 1, 700]), (128, 2, 1, [2500]), (64, 3, 3, [100, 5000])])
def test_prompt_values_that_are_not_finite_reach_no_earlier_row(moe, dtype, dim, hq, hkv, lens):
    n = sum(lens)
    q = rnd(n, hq, dim, dtype=dtype, seed=1, std=2.0)
    k, v = rnd(n, hkv, dim, dtype=dtype, seed=2), rnd(n, hkv, dim, dtype=dtype, seed=3)
    first, m = starts(lens)[-2], lens[-1]
    bad = m - 70                      # with rows of its tile of 128 on both sides
    v2 = v.clone()
    v2[first + bad, 0] = float("nan")
    if hkv > 1:
        v2[first + bad, 1, 5] = float("inf")
    v2[first + bad + 20, 0, 7] = -float("inf")
    out = moe.attend_prompt(q, k, v2, ints(starts(lens)))
    g = hq // hkv
    for a, x in zip(starts(lens), lens):
        if a != first:
            check_rows(out, q, k, v, a, x, list(range(x)), dim ** -0.5)
    check_rows(out, q, k, v, first, m, sorted({*range(max(0, bad - 140), bad), *range(0, bad, 37)}), dim ** -0.5)
    assert bool(out[first + bad:first + m, :g].isnan().all())
    if hkv > 1:
        row = out[first + bad:first + m, g:2 * g]
        assert not bool(row[..., 5].isfinite().any())
        rest = [c for c in range(dim) if c != 5]
        clean = moe.attend_prompt(q, k, v, ints(starts(lens)))[first + bad:first + m, g:2 * g]
        assert bool(row[..., rest].isfinite().all()) and bool((row[..., rest].float() - clean[..., rest].float()).abs().max() < 2 ** -6)


# ------------------------------------------------------------------ waits that run out


@pytest.mark.parametrize("dim,heads,lens", [(64, 100, [700]), (128, 4, [100, 8092])])
def test_prompt_wait_that_runs_out(moe, dim, heads, lens):
    """A CTA (or pair) that never gets its next item: all its rows are NaN, the error word says so, other
    rows are what they are without, and the next call is good."""
    n = sum(lens)
    q, k, v = rnd(n, heads, dim, dtype=BF, seed=1), rnd(n, heads, dim, dtype=BF, seed=2), rnd(n, heads, dim, dtype=BF, seed=3)
    cu, err = ints(starts(lens)), ints([0])
    want = moe.attend_prompt(q, k, v, cu, error=err)
    assert int(err) == 0
    out = torch.full_like(q, 3.0)
    assert moe.lib().moe_debug_stall_attention(1) == moe.MOE_OK
    t = time.monotonic()
    moe.attend_prompt(q, k, v, cu, out=out, error=err)
    torch.cuda.synchronize()
    assert 1.5 < time.monotonic() - t < 4  # the limit is 2 s
    assert int(err) == 3  # MOE_DEVERR_TMA
    nan = torch.zeros(n, heads, dtype=torch.bool, device=DEV)
    for s, block, h in turns(lens, heads, SMS)[1][0]:
        a = starts(lens)[s]
        nan[a + 256 * block:min(a + 256 * (block + 1), a + lens[s]), h] = True
    assert nan.any() and not nan.all()
    assert bool(out[nan].isnan().all()) and torch.equal(out[~nan], want[~nan])
    err.zero_()
    assert torch.equal(moe.attend_prompt(q, k, v, cu, error=err), want) and int(err) == 0


@pytest.mark.parametrize("dim,group,scored", [(64, 2, True), (128, 16, False)])
def test_attend_wait_that_runs_out(moe, dim, group, scored):
    """Copies that never come as long as they should be: NaN, the error word, and the next call is good."""
    lens = [300, 0, 17, 2000]
    c = Cache(moe, lens, 2, dim, 16, BF)
    q = rnd(4, 2 * group, dim, dtype=BF, seed=5)
    err, score = ints([0]), torch.zeros(4, 2, 2000, device=DEV)
    want = moe.kv_attend(c.pool, q, c.table, c.lens, 2000, error=err)
    assert moe.lib().moe_debug_stall_attention(1) == moe.MOE_OK
    t = time.monotonic()
    out = moe.kv_attend(c.pool, q, c.table, c.lens, 2000, score=score if scored else None, error=err)
    torch.cuda.synchronize()
    assert 1.5 < time.monotonic() - t < 4
    assert int(err) == 3  # MOE_DEVERR_TMA
    for b, n in enumerate(lens):
        assert bool(out[b].isnan().all()) if n else torch.equal(out[b], torch.zeros_like(out[b]))
        assert bool((score[b, :, n:] == 0).all()) and (not scored or bool(score[b, :, :n].isnan().all()))
    err.zero_()
    assert torch.equal(moe.kv_attend(c.pool, q, c.table, c.lens, 2000, error=err), want) and int(err) == 0


# ------------------------------------------------------------------ several host threads


def test_calls_from_several_threads(moe):
    """Four host threads, each with a stream and buffers of its own, at the same time; the C calls are made
    without the interpreter's lock."""
    import ctypes
    import threading
    P, L = ctypes.c_void_p, moe.lib()
    sets = []
    for s in range(4):
        c = Cache(moe, [300 + 100 * s, 17], 2, 64, 16, FP, seed=s)
        q = rnd(2, 8, 64, dtype=FP, seed=5 + s)
        p = [rnd(400, h, 64, dtype=FP, seed=s + h) for h in (4, 2, 2)]
        want = moe.kv_attend(c.pool, q, c.table, c.lens), moe.attend_prompt(*p, ints([0, 400]))
        sets.append((c, q, p, ints([0, 400]), want))
    torch.cuda.synchronize()
    bad = []

    def work(c, q, p, cu, want):
        try:
            stream = torch.cuda.Stream()
            for _ in range(50):
                a = moe.kv_attend(c.pool, q, c.table, c.lens, stream=stream)
                b = moe.attend_prompt(*p, cu, stream=stream)
                with torch.cuda.stream(stream):
                    d = torch.zeros_like(p[0])
                r = [moe.Rows(x.data_ptr(), x.stride(0), x.stride(1)) for x in (*p, d)]
                if L.moe_attend_prompt(0, *r, P(cu.data_ptr()), 1, 400, 4, 2, 64, moe.MOE_F16, 0.125, None, P(stream.cuda_stream)):
                    bad.append("status")
                try:
                    moe.kv_attend(c.pool, q.float(), c.table, c.lens)
                    bad.append("not refused")
                except moe.MoEError:
                    pass
                stream.synchronize()
                if not (torch.equal(a, want[0]) and torch.equal(b, want[1]) and torch.equal(d, want[1])):
                    bad.append("differs")
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))

    threads = [threading.Thread(target=work, args=s) for s in sets]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    assert not bad, bad


# ------------------------------------------------------------------ the ends of the documented ranges


@pytest.mark.parametrize("scored", [False, True])
@pytest.mark.parametrize("most", [0, 1, 33])
def test_attend_batch_without_positions(moe, scored, most):
    c = Cache(moe, [0, 0, 0], 2, 64, 16, BF, more=1)
    q, score = rnd(3, 8, 64, dtype=BF, seed=5), torch.ones(3, 2, 40, device=DEV)
    out = moe.kv_attend(c.pool, q, c.table, c.lens, most, score=score if scored else None)
    assert not bool(out.any()) and bool((score == 1).all())


@pytest.mark.parametrize("dim,heads,group,scored", [(128, 1, 8, False), (128, 1, 12, True), (64, 2, 1, True)])
def test_attend_most_sequences(moe, dim, heads, group, scored):
    """8192 sequences, most of them empty or of one position: the longest table of starts in shared memory."""
    lens = [0 if i % 3 else i % 40 for i in range(8192)]
    c = Cache(moe, lens, heads, dim, 16, FP)
    q, score = rnd(8192, heads * group, dim, dtype=FP, seed=5), torch.zeros(8192, heads, 39, device=DEV)
    out = moe.kv_attend(c.pool, q, c.table, c.lens, 39, score=score if scored else None)
    for b in (0, 1, 3, 39, 2000, 4095, 4098, 8189, 8190, 8191):
        check_attend(out, score.double() if scored else None, q, c, b, dim ** -0.5)
    assert bool(out.isfinite().all())


def test_attend_most_query_heads(moe):
    c = Cache(moe, [100, 3], 1, 64, 16, BF)
    q, score = rnd(2, 1024, 64, dtype=BF, seed=5), torch.zeros(2, 1, 100, device=DEV)
    out = moe.kv_attend(c.pool, q, c.table, c.lens, 100, score=score)
    for b in range(2):
        check_attend(out, None, q, c, b, 0.125)
    assert abs(float(score.double().sum()) - 2048) < 2048 * 2.0 ** -12


@pytest.mark.parametrize("seqs", [1, 254, 255, 256, 257, 8192])
def test_store_and_load_of_many_sequences(moe, seqs):
    lens = [(i * 7) % 4 for i in range(seqs)]
    lens[-1] = 3
    start = [(i * 5) % 30 for i in range(seqs)]
    n = sum(lens)
    k, v = rnd(n, 1, 64, dtype=BF, seed=1), rnd(n, 1, 64, dtype=BF, seed=2)
    table = tables(seqs, 3)
    pool = moe.kv_pool(table.numel(), 16, 1, 64)
    err = ints([0])
    moe.kv_store(pool, k, v, table, ints(starts(lens)), ints(start), error=err)
    gk, gv = moe.kv_load(pool, table, ints(starts(lens)), ints(start), n, F32, error=err)
    assert int(err) == 0 and torch.equal(gk.double(), quantised(k)) and torch.equal(gv.double(), quantised(v))


def test_large_pages_and_many_kv_heads(moe):
    lens = [5000, 1, 4096]
    c = Cache(moe, lens, 40, 64, 4096, FP)
    q = rnd(3, 80, 64, dtype=FP, seed=5)
    out = moe.kv_attend(c.pool, q, c.table, c.lens, 5000)
    for b in range(3):
        check_attend(out, None, q, c, b, 0.125)


@pytest.mark.parametrize("seqs", [31, 32, 33, 8192])
def test_prompt_many_sequences(moe, seqs):
    lens = [(i * 3) % 5 for i in range(seqs)]
    lens[seqs // 2] = 700
    n = sum(lens)
    q, k, v = rnd(n, 4, 64, dtype=FP, seed=1), rnd(n, 1, 64, dtype=FP, seed=2), rnd(n, 1, 64, dtype=FP, seed=3)
    out = moe.attend_prompt(q, k, v, ints(starts(lens)))
    cu = starts(lens)
    for s in sorted({0, 1, seqs // 2 - 1, seqs // 2, seqs // 2 + 1, seqs - 2, seqs - 1}):
        if lens[s]:
            check_rows(out, q, k, v, cu[s], lens[s], list(range(lens[s])), 0.125)
    assert bool(out.isfinite().all())


def test_graphs_of_two_streams_at_once(moe):
    """Two captured steps, each with buffers of its own, replayed on two streams without waiting in between."""
    def step(seed):
        c = Cache(moe, [700 + seed, 33], 2, 64, 16, FP, seed=seed, more=8)
        q, score = rnd(2, 8, 64, dtype=FP, seed=5 + seed), torch.zeros(2, 2, 720, device=DEV)
        p = [rnd(300, h, 64, dtype=FP, seed=seed + h) for h in (4, 2, 2)]
        cu, out_table = ints([0, 300]), tables(2, 4, first=c.table.numel())
        # everything the step allocates is made in here
        def run():
            score.zero_()
            o = moe.kv_attend(c.pool, q, c.table, c.lens, 720, score=score)
            n, kept, s = moe.kv_evict(c.pool, c.table, c.lens, 720, score, 50, 9, out_table)
            k, v = moe.kv_load(c.pool, out_table, ints_cu, None, 83, FP)
            return o, n, kept, s, k, v, moe.attend_prompt(*p, cu)
        ints_cu = ints([0, 50, 83])
        return run
    runs = [step(1), step(4)]
    want = [[x.clone() for x in r()] for r in runs]
    torch.cuda.synchronize()
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for r in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = r()
        graphs.append((g, got))
    for _ in range(30):
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for (_, got), w in zip(graphs, want):
        assert all(torch.equal(x, y) for x, y in zip(got, w))
