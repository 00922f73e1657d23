"""The paged serving calls on a machine without a GPU: sizes, and every refusal that is made
before anything is enqueued (the pointers are never followed)."""
import ctypes as C

import pytest

from token_recurrent_decoding_b200 import rlt

PTR = 1 << 20  # a 16- and 256-byte aligned address that no call may follow


def _cache(**kw):
    f = dict(pages=PTR, scales=None, n_pages=8, page_size=16, n_kv_heads=2, head_dim=64, dtype=1,
             kind=0)
    f.update(kw)
    return rlt.rlt_paged_kv(*(f[n] for n, _ in rlt.rlt_paged_kv._fields_))


def _rows(**kw):
    f = dict(page_table=PTR, table_width=4, cu_rows=PTR, kv_len=PTR, n=2, rows=0, status=None)
    f.update(kw)
    return rlt.rlt_paged_rows(*(f[n] for n, _ in rlt.rlt_paged_rows._fields_))


def _append(c, r, k=PTR, v=PTR, ld=128):
    return rlt._lib().rlt_paged_append(C.byref(c), C.byref(r), k, v, ld, None)


def _read(c, r, k=PTR, v=PTR, ld=128):
    return rlt._lib().rlt_paged_read(C.byref(c), C.byref(r), k, v, ld, None)


def _attend(c, r, q=PTR, ldq=128, heads=2, max_rows=4, max_len=64, window=0, out=PTR, ldo=128,
            lse=None, ws=PTR, nbytes=1 << 30):
    return rlt._lib().rlt_attend_paged(C.byref(c), C.byref(r), q, ldq, heads, max_rows, max_len,
                                       window, out, ldo, lse, ws, nbytes, None)


BAD_CACHES = [(dict(pages=None), 1), (dict(pages=PTR + 8), 1), (dict(n_pages=0), 1),
              (dict(page_size=0), 1), (dict(page_size=24), 1), (dict(page_size=2048), 1),
              (dict(n_kv_heads=0), 1), (dict(head_dim=48), 2), (dict(head_dim=256), 2),
              (dict(dtype=2), 1), (dict(kind=2), 1), (dict(kind=1), 1),
              (dict(kind=1, scales=PTR + 4), 1)]
BAD_ROWS = [dict(page_table=None), dict(cu_rows=None), dict(kv_len=None), dict(table_width=0),
            dict(n=0), dict(n=2049), dict(rows=-1)]


@pytest.mark.parametrize("call", [_append, _read, _attend])
def test_bad_caches_and_rows_are_refused(call):
    assert call(_cache(), _rows()) == 0  # no rows: nothing to do, nothing enqueued
    for kw, status in BAD_CACHES:
        assert call(_cache(**kw), _rows(rows=1)) == status, kw
    for kw in BAD_ROWS:
        assert call(_cache(), _rows(**{"rows": 1, **kw})) == 1, kw


@pytest.mark.parametrize("call", [_append, _read])
def test_bad_dense_rows_are_refused(call):
    r = _rows(rows=1)
    for kw in (dict(k=None), dict(v=None), dict(k=PTR + 2), dict(v=PTR + 8), dict(ld=127),
               dict(ld=130), dict(ld=-128)):
        assert call(_cache(), r, **kw) == 1, kw
    assert call(_cache(dtype=0), r, ld=130) == 1


def test_bad_attention_arguments_are_refused():
    r = _rows(rows=1)
    for kw in (dict(q=None), dict(out=None), dict(q=PTR + 8), dict(out=PTR + 4), dict(ldq=64),
               dict(ldo=132), dict(heads=3), dict(heads=0), dict(max_rows=-1), dict(max_len=-1),
               dict(window=-1), dict(ws=None), dict(ws=PTR + 16), dict(lse=PTR + 2),
               dict(max_len=1 << 30)):
        assert _attend(_cache(), r, **kw) == 1, kw
    assert _attend(_cache(), r, nbytes=0) == 4
    assert _attend(_cache(), r, max_rows=0) == 0


def test_attention_workspace_sizes():
    f = rlt._lib().rlt_attend_paged_workspace_bytes
    c = _cache()
    size = lambda n, heads, rows, mr, ml, cc=c: f(C.byref(cc), n, heads, rows, mr, ml)
    assert size(0, 2, 4, 4, 64) == 0 and size(1, 3, 4, 4, 64) == 0
    assert size(1, 2, -1, 4, 64) == 0 and size(2049, 2, 4, 4, 64) == 0
    assert size(1, 2, 4, 4, 64, _cache(head_dim=48)) == 0
    short = size(4, 2, 4, 1, 200)
    assert 0 < short < size(4, 2, 4, 1, 2000) <= size(4, 2, 4, 1, 20000)
    # a few splits of every row at most, and no more than the rule makes for long chunks
    assert size(1, 2, 1 << 16, 1 << 16, 1 << 18) < (1 << 16) * 2 * 66 * 4 * 2


def test_paged_rows_beyond_the_limits():
    lib = rlt._lib()
    assert lib.rlt_attend_paged_workspace_bytes(C.byref(_cache()), 1, 2, 1 << 28, 1, 64) == 0


def _verify(target=PTR, ts=64, tp=8, draft=PTR, ds=64, dp=8, tokens=PTR, lens=None, n=2, k=3,
            vocab=8, tau=1.0, u=PTR, out=PTR, counts=PTR, ws=PTR, nbytes=1 << 30):
    return rlt._lib().rlt_verify(target, ts, tp, draft, ds, dp, tokens, lens, n, k, vocab, tau, u,
                                 out, counts, ws, nbytes, None)


def test_bad_verifications_are_refused():
    for kw in (dict(target=None), dict(tokens=None), dict(u=None), dict(out=None),
               dict(counts=None), dict(ws=None), dict(ws=PTR + 8), dict(n=0), dict(k=-1),
               dict(k=33), dict(vocab=0), dict(tau=-1.0), dict(tau=float("nan")),
               dict(tau=float("inf")), dict(ts=-1), dict(dp=-1), dict(n=65536)):
        assert _verify(**kw) == 1, kw
    assert _verify(nbytes=0) == 4
    f = rlt.verify_workspace_bytes
    assert f(0, 1, 8) == 0 and f(1, 33, 8) == 0 and f(1, 1, 0) == 0
    assert 0 < f(2, 4, 32768) < f(4, 4, 32768) < f(4, 4, 131072)
