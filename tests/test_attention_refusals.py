"""The attention entry points refuse, before any device call, what they cannot do; their
structures have the header's layout.  No GPU: the addresses only have to look right."""
import ctypes
import os
import subprocess

import pytest

import expert_cache_host_router_b200 as moe
from expert_cache_host_router_b200 import build

P = 1 << 20  # an aligned address that nothing here reads


@pytest.fixture(scope="module")
def lib():
    build.build()
    return moe.lib()


def pool(**kw):
    d = dict(pool_dev=P, n_pages=8, n_kv_heads=2, head_dim=128, page_tokens=64, device=0, error_dev=None)
    d.update(kw)
    return moe.KvPool(*[d[n] for n, _ in moe.KvPool._fields_])


def table(**kw):
    d = dict(table_dev=P, n_seqs=3, width=4, row_stride=4)
    d.update(kw)
    return moe.KvTable(*[d[n] for n, _ in moe.KvTable._fields_])


def rows(data_dev=P, token_stride=256, head_stride=128):
    return moe.Rows(data_dev, token_stride, head_stride)


INVALID, UNSUPPORTED = moe.MOE_ERR_INVALID, moe.MOE_ERR_UNSUPPORTED
POOLS = [(dict(pool_dev=None), INVALID), (dict(pool_dev=P + 8), INVALID), (dict(n_pages=0), INVALID),
         (dict(n_kv_heads=0), INVALID), (dict(n_kv_heads=1025), UNSUPPORTED), (dict(head_dim=0), INVALID),
         (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=256), UNSUPPORTED), (dict(page_tokens=0), INVALID),
         (dict(page_tokens=24), UNSUPPORTED), (dict(device=-1), INVALID), (dict(device=64), INVALID)]
TABLES = [(dict(table_dev=None), INVALID), (dict(n_seqs=-1), INVALID), (dict(n_seqs=8193, width=1), UNSUPPORTED),
          (dict(width=0), INVALID), (dict(row_stride=3), INVALID), (dict(width=2 ** 26, row_stride=2 ** 26), UNSUPPORTED)]


@pytest.mark.parametrize("bad", [("pool", *b) for b in POOLS] + [("table", *b) for b in TABLES])
def test_every_cache_call_checks_pool_and_table(lib, bad):
    which, kw, status = bad
    c, t = (pool(**kw), table()) if which == "pool" else (pool(), table(**kw))
    s, n = moe.KvScore(P, 512, 256), ctypes.c_size_t()
    assert lib.moe_kv_store(c, t, P, P, rows(), rows(), 5, 0, None) == status
    assert lib.moe_kv_load(c, t, P, P, rows(), rows(), 5, 0, None) == status
    assert lib.moe_kv_attend(c, t, P, 100, rows(), 8, 0, 1.0, rows(), None, P, 1 << 40, None) == status
    assert lib.moe_kv_attend_workspace(c, t, 8, 100, 0, n) == status
    assert lib.moe_kv_evict(c, t, P, 100, s, 16, 4, table(table_dev=2 * P), 3 * P, P, P, None) == status
    if which == "table":
        assert lib.moe_kv_evict(c, table(), P, 100, s, 16, 4, t, 3 * P, P, P, None) == status


def test_rows_calls(lib):
    c, t = pool(), table()
    for f in (lib.moe_kv_store, lib.moe_kv_load):
        for args in ((None, P, rows(), rows(), 5, 0), (P, P, rows(data_dev=None), rows(), 5, 0), (P, P, None, rows(), 5, 0),
                     (P, P, rows(), None, 5, 0), (P, P, rows(), rows(), -1, 0), (P, P, rows(), rows(), 5, 3),
                     (P, P, rows(), rows(), 5, -1), (P, P, rows(data_dev=P + 1), rows(), 5, 0),
                     (P, P, rows(), rows(data_dev=P + 2), 5, moe.MOE_F32)):
            assert f(c, t, *args, None) == INVALID, args
        assert f(None, t, P, P, rows(), rows(), 5, 0, None) == INVALID
        assert f(c, None, P, P, rows(), rows(), 5, 0, None) == INVALID
        assert f(c, t, P, P, rows(), rows(), 2 ** 31 - 1, 0, None) == UNSUPPORTED
        assert f(c, t, P, None, rows(), rows(), 0, 0, None) == moe.MOE_OK  # nothing to do
        assert f(c, table(n_seqs=0), P, None, rows(), rows(), 5, 0, None) == moe.MOE_OK
    for bad in (rows(token_stride=0), rows(head_stride=0)):  # rows that are written need places of their own
        assert lib.moe_kv_load(c, t, P, P, bad, rows(), 5, 0, None) == INVALID
        assert lib.moe_kv_load(c, t, P, P, rows(), bad, 5, 0, None) == INVALID


def test_attend(lib):
    c, t = pool(), table()

    def call(lens=P, most=100, q=None, hq=8, dtype=0, scale=1.0, out=None, score=None, ws=P, size=1 << 40):
        return lib.moe_kv_attend(c, t, lens, most, q or rows(), hq, dtype, scale, out or rows(), score, ws, size, None)

    for kw in (dict(lens=None), dict(most=-1), dict(hq=0), dict(hq=7), dict(dtype=moe.MOE_F32), dict(dtype=9),
               dict(scale=0.0), dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")),
               dict(q=rows(data_dev=None)), dict(out=rows(data_dev=None)), dict(q=rows(data_dev=P + 1)),
               dict(out=rows(data_dev=P + 1)), dict(score=moe.KvScore(None, 8, 8)),
               dict(score=moe.KvScore(P, 0, 100)), dict(score=moe.KvScore(P, 200, 0)), dict(out=rows(token_stride=0)),
               dict(out=rows(head_stride=0))):
        assert call(**kw) == INVALID, kw
    assert call(hq=2 * 1025) == UNSUPPORTED and call(most=2 ** 31 - 1) == UNSUPPORTED
    assert lib.moe_kv_attend_workspace(c, t, 8, 100, 0, None) == INVALID
    assert lib.moe_kv_attend_workspace(c, t, 8, -1, 0, ctypes.c_size_t()) == INVALID
    assert lib.moe_kv_attend_workspace(pool(n_kv_heads=1024), table(n_seqs=8192), 1024, 2 ** 30, 0, ctypes.c_size_t()) == UNSUPPORTED


def test_evict(lib):
    c, t, o, s = pool(), table(), table(table_dev=2 * P), moe.KvScore(P, 512, 256)

    def call(lens=P, most=100, score=s, keep=16, recent=4, out=o, out_lens=3 * P, kept=P, out_score=4 * P):
        return lib.moe_kv_evict(c, t, lens, most, score, keep, recent, out, out_lens, kept, out_score, None)

    for kw in (dict(lens=None), dict(most=-1), dict(score=None), dict(score=moe.KvScore(None, 1, 1)), dict(keep=0),
               dict(recent=-1), dict(recent=17), dict(out=table(table_dev=P)), dict(out=table(table_dev=2 * P, n_seqs=2)),
               dict(keep=257), dict(out_lens=P), dict(out_lens=None), dict(kept=None), dict(out_score=P)):
        assert call(**kw) == INVALID, kw
    assert call(most=2 ** 31 - 1) == UNSUPPORTED


def test_prompt(lib):
    def call(dev=0, q=None, k=None, v=None, out=None, cu=P, b=2, n=100, hq=4, hkv=2, dim=64, dtype=0, scale=1.0):
        r = rows
        return lib.moe_attend_prompt(dev, q or r(), k or r(), v or r(), out or r(), cu, b, n, hq, hkv, dim, dtype, scale, None, None)

    for kw in (dict(dev=-1), dict(dev=64), dict(q=rows(None)), dict(k=rows(None)), dict(v=rows(None)), dict(out=rows(None)),
               dict(cu=None), dict(b=-1), dict(n=-1), dict(hq=0), dict(hkv=0), dict(hq=3), dict(dtype=2), dict(scale=0.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(out=rows(P + 1)), dict(out=rows(P, 0, 64)),
               dict(out=rows(P, 256, 0))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(dim=32), dict(dim=256), dict(b=8193), dict(q=rows(P + 8)), dict(k=rows(P, 12, 64)), dict(v=rows(P, 64, 4)),
               dict(q=rows(P, -64, 64)), dict(k=rows(P, 128, 0)), dict(v=rows(P, 0, 64)), dict(n=2 ** 31 - 1)):
        assert call(**kw) == UNSUPPORTED, kw
    assert call(n=0) == moe.MOE_OK and call(b=0) == moe.MOE_OK


def test_binding_refuses_wrong_tensors():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(moe.MoEError):
        moe.kv_store(torch.zeros(2, 2, 1, 18 * 64, dtype=torch.uint8), x, x, i[None], i)
    with pytest.raises(moe.MoEError):
        moe.attend_prompt(x, x, x, i)
    for bad in (dict(page_tokens=24), dict(page_tokens=0), dict(head_dim=80)):
        with pytest.raises(moe.MoEError):
            moe.kv_pool(**{**dict(n_pages=2, page_tokens=16, n_kv_heads=1, head_dim=64), **bad})


def test_struct_layouts(tmp_path):
    structs = {"moe_kv_pool": moe.KvPool, "moe_kv_table": moe.KvTable, "moe_rows": moe.Rows, "moe_kv_score": moe.KvScore}
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "moe_cache.h"', "int main(void) {"]
    for c, cls in structs.items():
        lines.append(f'  printf("%zu\\n", sizeof({c}));')
        lines += [f'  printf("%zu\\n", offsetof({c}, {f}));' for f, _ in cls._fields_]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines + ["  return 0;", "}", ""]))
    inc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include")
    subprocess.check_call(["gcc", "-std=c11", f"-I{inc}", str(src), "-o", str(exe)])
    want = []
    for cls in structs.values():
        want.append(ctypes.sizeof(cls))
        want += [getattr(cls, f).offset for f, _ in cls._fields_]
    assert [int(x) for x in subprocess.check_output([str(exe)], text=True).split()] == want
