"""Corners of the attention operators: packed prompts of which a pair's second CTA has no key tile.

Against 64 bits, with the tolerances that tests/test_gpu_attention.py derives."""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_attention import BF, DEV, FP, Cache, check_attend, half, ints, moe, quantised, rnd, starts, tables  # noqa: E402,F401
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
