"""The paged serving bindings' own checks on a machine without a GPU, on stand-ins of tensors: sizes
that the C ABI's 32-bit ints do not hold are refused, not cut."""
import pytest
import torch

from token_recurrent_decoding_b200 import rlt

BEYOND = 2 ** 32 + 4  # cut to 32 bits: 4


class Stand:
    """What the checks ask of a contiguous tensor on GPU 0."""

    def __init__(self, *shape, dtype=torch.int32):
        self.shape, self.dtype, self.device, self.is_cuda = shape, dtype, "cuda:0", True

    def dim(self):
        return len(self.shape)

    def size(self, i):
        return self.shape[i]

    def stride(self):
        out, s = [], 1
        for n in reversed(self.shape):
            out.append(s)
            s *= n
        return tuple(reversed(out))

    def numel(self):
        n = 1
        for x in self.shape:
            n *= x
        return n

    is_contiguous = lambda self: True  # noqa: E731
    get_device = lambda self: 0  # noqa: E731
    data_ptr = lambda self: 1 << 20  # noqa: E731


def rows(*shape):
    return Stand(*shape, dtype=torch.bfloat16)


@pytest.fixture
def cache(monkeypatch):
    rlt._lazy_torch()
    monkeypatch.setattr(rlt, "_launch", lambda *a: pytest.fail("launched"))
    return rlt.PagedKV(rows(8, 2, 2, 16, 64))


def _attend(cache, q=None, table=None, max_rows=4, max_len=64, window=0, n_rows=4):
    q = q or rows(n_rows, 4, 64)
    return rlt.attend_paged(q, cache, table or Stand(1, 4), Stand(2), Stand(1), max_rows, max_len,
                            out=q, window=window, workspace=Stand(1 << 20, dtype=torch.uint8))


def test_the_call_that_the_others_vary_is_made(cache, monkeypatch):
    made = []
    monkeypatch.setattr(rlt, "_launch", lambda *a: made.append(a))
    _attend(cache)
    k = rows(4, 2, 64)
    rlt.paged_append(cache, Stand(1, 4), k, k, Stand(2), Stand(1))
    assert len(made) == 2


def test_sizes_beyond_32_bits_are_refused(cache):
    for kw in (dict(max_rows=BEYOND), dict(max_len=BEYOND), dict(window=BEYOND),
               dict(window=-BEYOND), dict(max_rows=-1), dict(max_len=-BEYOND),
               dict(table=Stand(1, BEYOND)), dict(n_rows=BEYOND), dict(q=rows(4, BEYOND, 64))):
        with pytest.raises(rlt.RLTError):
            _attend(cache, **kw)
    k = rows(BEYOND, 2, 64)
    for fn in (lambda: rlt.paged_append(cache, Stand(1, 4), k, k, Stand(2), Stand(1)),
               lambda: rlt.paged_read(cache, Stand(1, BEYOND), Stand(2), Stand(1), rows(4, 2, 64),
                                      rows(4, 2, 64))):
        with pytest.raises(rlt.RLTError):
            fn()
    for args in ((BEYOND, 4, 4, 4, 64), (1, 4, BEYOND, 4, 64), (1, 4, 4, 4, BEYOND)):
        assert rlt.attend_paged_workspace_bytes(cache, *args) == 0
    assert rlt.attend_paged_workspace_bytes(cache, 1, 4, 4, 4, 6400) > 0


def test_verifications_beyond_32_bits_are_refused(cache):
    f32 = lambda *s: Stand(*s, dtype=torch.float32)  # noqa: E731
    for n, V in ((BEYOND, 8), (2, BEYOND)):
        with pytest.raises(rlt.RLTError):
            rlt.verify(f32(n, 1, V), None, None, 1.0, f32(n, 1), tokens=Stand(n, 1),
                       counts=Stand(n), workspace=Stand(1 << 20, dtype=torch.uint8))
    assert rlt.verify_workspace_bytes(2, 1, BEYOND) == 0
    assert rlt.verify_workspace_bytes(BEYOND, 1, 8) == 0


def test_more_rows_than_blocks_can_number_are_refused():
    """The C ABI's own int holds them; the grid's size would not."""
    import ctypes as C
    c = rlt.rlt_paged_kv(1 << 20, None, 8, 16, 2, 64, 1, 0)
    for rows_ in (2 ** 31 - 1, 2 ** 30 + 1):
        r = rlt.rlt_paged_rows(1 << 20, 4, 1 << 20, 1 << 20, 2, rows_, None)
        for fn in (rlt._lib().rlt_paged_append, rlt._lib().rlt_paged_read):
            assert fn(C.byref(c), C.byref(r), 1 << 20, 1 << 20, 128, None) == 1
