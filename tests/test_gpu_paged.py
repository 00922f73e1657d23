"""The paged cache and the attention over it, on the GPU, against float64 on the CPU."""
import math

import numpy as np
import pytest
import torch

from paged_cases import BF16, E4, F32, Case, attend64, attend_bound, quantised
from token_recurrent_decoding_b200 import rlt

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- the cache itself
def _special(x):
    """A few blocks with what rounds at a border, tiny, huge, zero and not finite."""
    f = x.view(-1)
    f[:32] = 0
    f[32:64] = 448.0 * torch.arange(1, 33) / 32
    f[64] = 448.5
    f[96] = 3e38
    f[128] = 1e-38
    f[160:192] = torch.tensor([1.0, 1.0625, 1.1875, 448.0] * 8)  # ties to even
    f[192] = math.inf
    f[224] = math.nan
    f[256] = 2.0 ** -130
    return x


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kind", [rlt.KV_PLAIN, rlt.KV_E4M3])
@pytest.mark.parametrize("dh,page,H", [(16, 16, 3), (32, 48, 2), (64, 16, 1), (128, 64, 2)])
def test_rows_written_and_read_back(dtype, kind, dh, page, H):
    rows, lens = [0, 5, 1, 0, 33, 17], [0, 9, 1, 4, 70, 17]
    c = Case(rows, lens, H=H, dh=dh, page=page, dtype=dtype, pad=3).device()
    wide = torch.randn((c.total, 2 * H + 1, dh), generator=c.g)
    _special(wide[5:30].view(-1)[: 20 * (2 * H + 1) * dh])
    wide = wide.to(dtype)
    dw = wide.cuda()
    k, v = dw[:, 1:1 + H], dw[:, 1 + H:]
    cache = rlt.PagedKV.empty(c.n_pages, page, H, dh, dtype, kind)
    cache.pages.view(torch.uint8).fill_(0x2a)
    if kind == rlt.KV_E4M3:
        cache.scales.fill_(99)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rlt.paged_append(cache, c.d_table, k, v, c.d_cu, c.d_len, status=status)
    ko, vo = (torch.full((c.total, H, dh), 7.0, dtype=dtype, device="cuda") for _ in range(2))
    rlt.paged_read(cache, c.d_table, c.d_cu, c.d_len, ko, vo, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    # the pages, byte by byte: the listed rows as float64 rounds them, all else as it was
    want = torch.full(cache.pages.shape, 0x2a, dtype=torch.uint8).expand(cache.pages.shape).clone()
    B, es = min(32, dh), torch.finfo(cache.pages.dtype).bits // 8
    want = torch.full((c.n_pages, H, 2, page, dh * es), 0x2a, dtype=torch.uint8)
    wsc = torch.full((c.n_pages, H, 2, page, dh // B), 99, dtype=torch.uint8)
    back = torch.full((2, c.total, H, dh), 7.0, dtype=torch.float64)
    r = 0
    for b, m in enumerate(rows):
        for i in range(m):
            p = lens[b] - m + i
            pg, sl = int(c.table[b, p // page]), p % page
            x = torch.stack([wide[r, 1:1 + H], wide[r, 1 + H:]], 1)  # [H][2][dh]
            if kind == rlt.KV_E4M3:
                val, byte = quantised(x.double().numpy())
                wsc[pg, :, :, sl] = torch.from_numpy(byte)
                y = val.reshape(H, 2, -1, B) / 2.0 ** (byte.astype(float) - 127)[..., None]
                y = np.where(byte[..., None] == 255, 0.0, y).reshape(H, 2, dh)
                want[pg, :, :, sl] = torch.from_numpy(y).float().to(E4).view(torch.uint8)
                back[:, r] = torch.from_numpy(val).permute(1, 0, 2)
            else:
                want[pg, :, :, sl] = x.contiguous().view(torch.uint8)
                back[:, r] = x.double().permute(1, 0, 2)
            r += 1
    got = cache.pages.view(torch.uint8).reshape(want.shape).cpu()
    if kind == rlt.KV_E4M3:
        # zeros may carry a sign
        fix = lambda t: torch.where(t == 0x80, 0, t)  # noqa: E731
        assert torch.equal(fix(got), fix(want))
        assert torch.equal(cache.scales.cpu(), wsc)
    else:
        assert torch.equal(got, want)
    for got, ref in zip((ko, vo), back):
        got = got.double().cpu()
        assert torch.equal(got.isnan(), ref.isnan())
        assert torch.equal(got.nan_to_num(0.0, 1e300, -1e300), ref.nan_to_num(0.0, 1e300, -1e300))


@pytest.mark.parametrize("kind", [rlt.KV_PLAIN, rlt.KV_E4M3])
def test_pages_and_rows_that_do_not_exist(kind):
    c = Case([4, 4, 4, 4], [20, 20, 20, 3], H=2, dh=32, page=16, dtype=F32).device()
    cache = rlt.PagedKV.empty(c.n_pages, 16, 2, 32, F32, kind)
    cache.pages.view(torch.uint8).fill_(1)
    if kind == rlt.KV_E4M3:
        cache.scales.fill_(127)
    before = cache.pages.view(torch.uint8).clone()
    x = torch.randn((16, 2, 32), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    table = c.d_table.clone()
    table[0, 1], table[1, 1], table[2, 1] = c.n_pages, -1, 1 << 30
    # sequence 3 has four rows and three positions: its first row lies before position 0
    rlt.paged_append(cache, table, x, x, c.d_cu, c.d_len, status=status)
    assert int(status) == rlt.PAGED_BAD_PAGE
    out = torch.full_like(x, 5.0)
    out2 = out.clone()
    status.zero_()
    rlt.paged_read(cache, table, c.d_cu, c.d_len, out, out2, status=status)
    assert int(status) == rlt.PAGED_BAD_PAGE
    assert (out[:13] == 0).all() and (out[13:] != 0).any() and not (out[13:] == 5).any()
    page = int(c.table[3, 0])
    keep = [p for p in range(c.n_pages) if p != page]
    assert torch.equal(cache.pages.view(torch.uint8)[keep], before[keep])
    # positions beyond the table, rows that are none of the call
    status.zero_()
    rlt.paged_append(cache, c.d_table, x, x, c.d_cu, torch.full_like(c.d_len, 1 << 30),
                     status=status)
    assert int(status) == rlt.PAGED_BAD_PAGE
    for cu in ([0, 4, 2, 12, 16], [-3, 4, 8, 12, 16], [0, 4, 8, 12, 99]):
        status.zero_()
        bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
        kept = cache.pages.view(torch.uint8).clone()
        rlt.paged_append(cache, c.d_table, x, x, bad, c.d_len, status=status)
        assert int(status) == rlt.PAGED_BAD_ROWS, cu
        assert torch.equal(cache.pages.view(torch.uint8), kept)
        mine = torch.full_like(x, 5.0)
        rlt.paged_read(cache, c.d_table, bad, c.d_len, mine, mine.clone())
        assert (mine == 5).all()


# --------------------------------------------------------------- the attention
def _check(c, heads, window=0, scale=1.0, lse=True, max_rows=None, max_len=None, stream=None):
    q = c.queries(heads, scale)
    dq = q.cuda()
    assert dq.stride() != q.contiguous().stride() or c.total < 2 or True
    out = torch.full((c.total, heads + 1, c.dh), 9.0, dtype=c.dtype, device="cuda")[:, :heads]
    l = torch.full((c.total, heads), 9.0, device="cuda") if lse else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rlt.attend_paged(dq, c.cache, c.d_table, c.d_cu, c.d_len, max_rows or max(c.rows),
                     max_len or max(c.lens), out=out, lse=l, window=window, status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    got = out.double().cpu()
    end = int(c.cu[-1])
    assert (got[end:] == 9.0).all()
    worst = err2 = ref2 = 0.0
    for b, m in enumerate(c.rows):
        lo = int(c.cu[b])
        ref, rl, mass, size = attend64(q[lo:lo + m].double(), c.kv[b], c.lens[b], window)
        bound = attend_bound(ref, mass, size, c.dh, c.dtype)
        err = (got[lo:lo + m] - ref).abs()
        assert torch.isfinite(got[lo:lo + m]).all()
        worst = max([worst] + (err / bound).flatten().tolist())
        err2, ref2 = err2 + float((err ** 2).sum()), ref2 + float((ref ** 2).sum())
        if lse:
            g = l[lo:lo + m].double().cpu()
            assert torch.equal(torch.isinf(g), torch.isinf(rl))
            fin = torch.isfinite(rl)
            lb = size * (c.dh + 8) * 2.0 ** -23 + 512 * 2.0 ** -23 + rl.abs() * 2.0 ** -22
            assert ((g - rl).abs()[fin] <= lb[fin]).all()
    assert worst <= 1.0, worst
    # in the norm the roundings of fp32 have random signs: sqrt(512) of them, not 512
    if c.dtype == F32 and ref2 > 0:
        assert math.sqrt(err2 / ref2) <= 1e-5
    return got


CHUNKS = [  # rows, lengths
    ([1], [1]),
    ([1, 1, 1, 1], [1, 2, 15, 16]),
    ([1, 1, 1], [17, 300, 1023]),
    ([5, 5, 2], [5, 64, 700]),
    ([0, 16, 0, 17, 1], [40, 16, 0, 33, 500]),
    ([40, 3, 100], [40, 90, 612]),
]


@pytest.mark.parametrize("kind", ["bf16", "f32", "bf16e4", "f32e4"])
@pytest.mark.parametrize("rows,lens", CHUNKS)
@pytest.mark.parametrize("dh", [16, 32, 64, 128])
def test_attention(kind, rows, lens, dh):
    H, heads = (2, 2) if dh >= 64 else (1, 3)
    c = Case(rows, lens, H=H, dh=dh, page=16, dtype=F32 if kind[0] == "f" else BF16,
             e4=kind.endswith("e4"), seed=len(rows) + dh, pad=2).device()
    _check(c, heads)


@pytest.mark.parametrize("kind", ["bf16", "f32", "bf16e4", "f32e4"])
@pytest.mark.parametrize("group,page,window", [(1, 48, 0), (4, 16, 40), (3, 32, 1), (8, 64, 300),
                                               (7, 16, 17), (2, 1024, 0)])
def test_shared_heads_pages_and_windows(kind, group, page, window):
    c = Case([1, 4, 70, 9], [200, 4, 260, 641], H=2, dh=64, page=page,
             dtype=F32 if kind[0] == "f" else BF16, e4=kind.endswith("e4"), seed=group).device()
    _check(c, 2 * group, window=window)


@pytest.mark.parametrize("kind", ["bf16", "f32", "bf16e4"])
def test_sharp_scores_and_long_sequences(kind):
    """Scores of tens: one key takes a row; and splits of a few thousand keys."""
    c = Case([2, 1], [5000, 3333], H=1, dh=128, page=64, dtype=F32 if kind[0] == "f" else BF16,
             e4=kind.endswith("e4"), seed=3).device()
    _check(c, 2, scale=6.0)


@pytest.mark.parametrize("value_scale", [1e6, 1e30, 1e-30])
@pytest.mark.parametrize("dtype,m,dh", [(BF16, 2, 128), (BF16, 60, 128), (F32, 3, 64),
                                        (BF16, 2, 32)])
def test_scales_far_from_one(value_scale, dtype, m, dh):
    c = Case([m, 1], [90 + m, 33], H=2, dh=dh, page=16, dtype=dtype, e4=True, seed=11,
             value_scale=value_scale).device()
    _check(c, 2)


@pytest.mark.parametrize("kind", ["bf16", "bf16e4"])
@pytest.mark.parametrize("dh,m,lens", [(128, 40, [9000, 700]), (64, 300, [9100, 4300]),
                                       (128, 33, [128, 40])])
def test_long_sequences_and_wide_tiles(kind, dh, m, lens):
    """Split ranges, streams of key tiles (an odd number of them, one of them) and tiles whose
    second half has few rows or none."""
    c = Case([m, 35], lens, H=1, dh=dh, page=128, e4=kind.endswith("e4"), seed=12).device()
    _check(c, 1, window=0 if dh == 128 else 8000)


@pytest.mark.parametrize("kind", ["bf16", "f32", "bf16e4"])
@pytest.mark.parametrize("m", [3, 90])
def test_what_lies_in_unseen_places_does_not_matter(kind, m):
    """NaN in stale pages, behind the sequence, and in keys and values that only later rows see."""
    e4 = kind.endswith("e4")
    c = Case([m, 1], [130 + m, 77], H=2, dh=64, page=32, dtype=F32 if kind[0] == "f" else BF16,
             e4=e4, seed=5, stale=math.nan)
    L = c.lens[0]
    for kv in (0, 1):  # the last token's key and value
        pg, sl = int(c.table[0, (L - 1) // 32]), (L - 1) % 32
        if e4:
            c.scales[pg, 0, kv, sl] = 255
            c.pages.view(torch.uint8)[pg, 0, kv, sl] = 0
        else:
            c.pages[pg, 0, kv, sl] = math.nan
    c.device()
    q = c.queries(2)
    out = rlt.attend_paged(q.cuda(), c.cache, c.d_table, c.d_cu, c.d_len, m, L).double().cpu()
    ref, _, mass, size = attend64(q[:m].double(), c.kv[0], L, 0)
    ok = torch.ones((m, 2), dtype=torch.bool)
    ok[m - 1, 0] = False  # the row and head that see them
    err = (out[:m] - ref).abs()
    assert torch.isfinite(out[:m][ok]).all() and torch.isnan(out[m - 1, 0]).all()
    assert (err[ok] <= attend_bound(ref, mass, size, 64, c.dtype)[ok]).all()
    assert torch.isfinite(out[m]).all()


@pytest.mark.parametrize("kind", ["bf16", "bf16e4"])
def test_keys_on_missing_pages_do_not_exist(kind):
    c = Case([2, 2], [64, 64], H=1, dh=64, page=16, e4=kind.endswith("e4"), seed=6).device()
    table = c.d_table.clone()
    table[0, 1] = c.n_pages + 7
    table[1, :] = -1
    q = c.queries(1)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lse = torch.zeros((4, 1), device="cuda")
    out = rlt.attend_paged(q.cuda(), c.cache, table, c.d_cu, c.d_len, 2, 64, lse=lse,
                           status=status).double().cpu()
    assert int(status) == rlt.PAGED_BAD_PAGE
    kv = torch.cat([c.kv[0][:16], c.kv[0][32:]])
    ref, _, mass, size = attend64(q[:2].double(), kv, 48, 0)
    assert ((out[:2] - ref).abs() <= attend_bound(ref, mass, size, 64, BF16)).all()
    assert (out[2:] == 0).all() and torch.isinf(lse[2:]).all()


def test_rows_before_the_first_position_and_bad_rows():
    c = Case([6, 1], [6, 20], H=1, dh=64, page=16, seed=7).device()
    q = c.queries(2).cuda()
    short = torch.tensor([4, 20], dtype=torch.int32, device="cuda")  # rows at positions -2, -1
    lse = torch.zeros((7, 2), device="cuda")
    out = rlt.attend_paged(q, c.cache, c.d_table, c.d_cu, short, 6, 20, lse=lse)
    assert (out[:2] == 0).all() and (lse[:2] == -math.inf).all()
    assert (out[2:] != 0).any(-1).all() and torch.isfinite(lse[2:]).all()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    for max_rows, max_len, kept in ((5, 20, slice(0, 6)), (6, 19, slice(6, 7))):
        mine = torch.full_like(out, 3.0)
        status.zero_()
        rlt.attend_paged(q, c.cache, c.d_table, c.d_cu, c.d_len, max_rows, max_len, out=mine,
                         status=status)
        assert int(status) == rlt.PAGED_BAD_ROWS and (mine[kept] == 3).all()
        assert not (mine == 3).all()
    for cu in ([0, 9, 7], [0, 7, 6], [-1, 6, 7]):
        mine = torch.full_like(out, 3.0)
        status.zero_()
        rlt.attend_paged(q, c.cache, c.d_table,
                         torch.tensor(cu, dtype=torch.int32, device="cuda"), c.d_len, 6, 20,
                         out=mine, status=status)
        assert int(status) & rlt.PAGED_BAD_ROWS and (mine == 3).all(), cu


@pytest.mark.parametrize("kind", ["bf16", "f32", "bf16e4"])
def test_a_row_does_not_depend_on_its_batch(kind):
    rows, lens = [1, 50, 5, 1, 200], [900, 333, 1500, 64, 700]
    c = Case(rows, lens, H=2, dh=64, page=32, dtype=F32 if kind[0] == "f" else BF16,
             e4=kind.endswith("e4"), seed=8).device()
    q = c.queries(4).cuda()
    out = rlt.attend_paged(q, c.cache, c.d_table, c.d_cu, c.d_len, 200, 1500)
    for b, m in enumerate(rows):
        lo = int(c.cu[b])
        cu = torch.tensor([0, m], dtype=torch.int32, device="cuda")
        one = rlt.attend_paged(q[lo:lo + m], c.cache, c.d_table[b:b + 1], cu, c.d_len[b:b + 1], m,
                               lens[b])
        assert torch.equal(one, out[lo:lo + m]), b


def test_captured_calls_follow_their_inputs():
    """Append, attend and read in one graph, replayed with other rows, lengths and pages, and two
    graphs that share a workspace replayed one after the other; a stream of its own."""
    c = Case([3, 40], [400, 555], H=2, dh=64, page=16, e4=True, seed=9).device()
    heads = 4
    side = torch.cuda.Stream()
    q = torch.zeros((43, heads, 64), dtype=BF16, device="cuda")
    k, v, ko, vo = (torch.zeros((43, 2, 64), dtype=BF16, device="cuda") for _ in range(4))
    outs = [torch.zeros_like(q) for _ in range(2)]
    work = torch.empty(rlt.attend_paged_workspace_bytes(c.cache, 2, heads, 43, 40, 600),
                       dtype=torch.uint8, device="cuda")

    def step(out):
        rlt.paged_append(c.cache, c.d_table, k, v, c.d_cu, c.d_len, stream=side)
        rlt.attend_paged(q, c.cache, c.d_table, c.d_cu, c.d_len, 40, 600, out=out, workspace=work,
                         stream=side)
        rlt.paged_read(c.cache, c.d_table, c.d_cu, c.d_len, ko, vo, stream=side)

    side.wait_stream(torch.cuda.current_stream())
    graphs = []
    for out in outs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step(out)
        graphs.append(graph)
    g = torch.Generator().manual_seed(1)
    for rows, lens in (([3, 40], [400, 555]), ([20, 1], [380, 512]), ([0, 33], [17, 600])):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=g))
        c.d_cu.copy_(torch.tensor([0, rows[0], sum(rows)]))
        c.d_len.copy_(torch.tensor(lens))
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for graph in graphs:
                graph.replay()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        n = sum(rows)
        want = rlt.attend_paged(q, c.cache, c.d_table, c.d_cu, c.d_len, 40, 600)
        assert torch.equal(outs[0][:n], want[:n]) and torch.equal(outs[1][:n], want[:n])
        ref = quantised(torch.stack([k, v], 2).double().cpu().numpy()[:n])[0]
        # positions from 560 on have no page: such rows read as zeros
        ref[[lens[b] - rows[b] + i >= 560 for b in (0, 1) for i in range(rows[b])]] = 0
        assert np.array_equal(ko[:n].double().cpu().numpy(), ref[:, :, 0])
        assert np.array_equal(vo[:n].double().cpu().numpy(), ref[:, :, 1])


def test_two_calls_at_once():
    c = Case([1, 1, 9], [3000, 2000, 1500], H=2, dh=128, page=64, seed=10).device()
    q = c.queries(4).cuda()
    want = rlt.attend_paged(q, c.cache, c.d_table, c.d_cu, c.d_len, 9, 3000)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = [rlt.attend_paged(q, c.cache, c.d_table, c.d_cu, c.d_len, 9, 3000, stream=s)
            for _ in range(5) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_tensors_that_do_not_fit_are_refused():
    c = Case([2], [40], H=2, dh=64, page=16).device()
    q = c.queries(4).cuda()
    call = lambda **kw: rlt.attend_paged(**{**dict(  # noqa: E731
        q=q, cache=c.cache, table=c.d_table, cu_rows=c.d_cu, kv_len=c.d_len, max_rows=2,
        max_len=40), **kw})
    for kw in (dict(q=q.float()), dict(q=q[:, :3]), dict(q=q[..., :32]), dict(q=q.cpu()),
               dict(table=c.d_table.long()), dict(table=c.d_table.cpu()), dict(cu_rows=c.d_len),
               dict(kv_len=c.d_len.long()), dict(lse=torch.zeros(2, 3, device="cuda")),
               dict(out=torch.zeros(2, 4, 64, device="cuda")), dict(window=-1),
               dict(workspace=torch.empty(8, dtype=torch.uint8, device="cuda")),
               dict(status=torch.zeros(1, device="cuda"))):
        with pytest.raises(rlt.RLTError):
            call(**kw)
    k = torch.zeros((2, 2, 64), dtype=BF16, device="cuda")
    for a, b in ((k.float(), k.float()), (k, k[:1]), (k[:, :1], k[:, :1]),
                 (k.transpose(1, 2), k.transpose(1, 2))):
        with pytest.raises(rlt.RLTError):
            rlt.paged_append(c.cache, c.d_table, a, b, c.d_cu, c.d_len)
    pages = torch.zeros((2, 2, 2, 16, 64), device="cuda")
    for args in ((pages.half(),), (pages.cpu(),), (pages[..., ::2],), (pages.to(E4),),
                 (pages, torch.zeros((2, 2, 2, 16, 2), dtype=torch.uint8, device="cuda")),
                 (pages.to(E4), torch.zeros((2, 2, 2, 16, 1), dtype=torch.uint8, device="cuda"))):
        with pytest.raises(rlt.RLTError):
            rlt.PagedKV(*args)


@pytest.mark.parametrize("kind,m", [("bf16", 2), ("bf16", 50), ("bf16e4", 50), ("f32", 2)])
def test_pages_behind_four_gigabytes(kind, m):
    """The sequence's pages are the last of a pool of more than 2^32 bytes (and elements, in 8 bits)."""
    e4, dtype, page, dh = kind.endswith("e4"), F32 if kind == "f32" else BF16, 1024, 128
    es = 1 if e4 else 4 if dtype == F32 else 2
    per_page = 2 * page * dh * es
    n_pages = 2 ** 32 // per_page + 64
    cache = rlt.PagedKV.empty(n_pages, page, 1, dh, dtype, rlt.KV_E4M3 if e4 else rlt.KV_PLAIN)
    L = 1500
    g = torch.Generator().manual_seed(1)
    kv = torch.randn((L, 1, 2, dh), generator=g).to(dtype)
    table = torch.tensor([[n_pages - 1, n_pages - 3]], dtype=torch.int32).cuda()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32).cuda()  # noqa: E731
    d = kv.cuda()
    rlt.paged_append(cache, table, d[:, :, 0], d[:, :, 1], i32(0, L), i32(L))
    held = torch.from_numpy(quantised(kv.double().numpy())[0]) if e4 else kv.double()
    ko, vo = (torch.empty((L, 1, dh), dtype=dtype, device="cuda") for _ in range(2))
    rlt.paged_read(cache, table, i32(0, L), i32(L), ko, vo)
    assert torch.equal(ko.double().cpu(), held[:, :, 0])
    assert torch.equal(vo.double().cpu(), held[:, :, 1])
    q = torch.randn((m, 1, dh), generator=g).to(dtype)
    out = rlt.attend_paged(q.cuda(), cache, table, i32(0, m), i32(L), m, L).double().cpu()
    ref, _, mass, size = attend64(q.double(), held, L, 0)
    assert ((out - ref).abs() <= attend_bound(ref, mass, size, dh, dtype)).all()


@pytest.mark.parametrize("kind", ["bf16", "f32", "bf16e4"])
def test_the_largest_batch(kind):
    """2048 sequences: the plan at its largest beside the largest tiles in shared memory; empty ones,
    one with enough rows for 128-row tiles, one with enough keys for splits."""
    n = 2048
    rows = [(i * 7) % 3 for i in range(n)]
    lens = [r + (i * 5) % 4 for i, r in enumerate(rows)]
    rows[1000], lens[1000] = 45, 60
    rows[2047], lens[2047] = 1, 700
    c = Case(rows, lens, H=1, dh=128, page=16, dtype=F32 if kind == "f32" else BF16,
             e4=kind.endswith("e4"), seed=13, pad=1).device()
    _check(c, 1)
    k = torch.zeros((c.total, 1, 128), dtype=c.dtype, device="cuda")
    rlt.paged_append(c.cache, c.d_table, k, k, c.d_cu, c.d_len)
    out, out2 = torch.ones_like(k), torch.ones_like(k)
    rlt.paged_read(c.cache, c.d_table, c.d_cu, c.d_len, out, out2)
    assert (out[:-1] == 0).all() and (out[-1] == 1).all() and (out2[:-1] == 0).all()
    bad = torch.zeros(n + 1, dtype=torch.int32, device="cuda")
    with pytest.raises(rlt.RLTError):
        rlt.paged_read(c.cache, torch.zeros((n + 1, 1), dtype=torch.int32, device="cuda"),
                       torch.zeros(n + 2, dtype=torch.int32, device="cuda"), bad, out, out2)


def test_a_first_call_may_be_captured():
    """In a process of its own: nothing of the library has run before the capture."""
    code = '''
import torch
from token_recurrent_decoding_b200 import rlt
cache = rlt.PagedKV.empty(8, 16, 2, 64, torch.bfloat16, rlt.KV_E4M3)
i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
table, cu, n = torch.arange(8, device="cuda").int()[None], i32(0, 40), i32(100)
x = torch.randn(40, 4, 64, device="cuda").bfloat16()
out = torch.zeros_like(x)
t = torch.randn(2, 3, 500, device="cuda")
u = torch.rand(2, 3, device="cuda")
d = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
work = torch.empty(rlt.attend_paged_workspace_bytes(cache, 1, 4, 40, 40, 100), dtype=torch.uint8,
                   device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    rlt.paged_append(cache, table, x[:, :2], x[:, 2:], cu, n)
    rlt.attend_paged(x, cache, table, cu, n, 40, 100, out=out, workspace=work)
    tokens, counts = rlt.verify(t, t[:, :2], d, 1.0, u)
cache.pages.view(torch.uint8).zero_()
cache.scales.fill_(127)
graph.replay()
torch.cuda.synchronize()
want = rlt.attend_paged(x, cache, table, cu, n, 40, 100)
assert torch.equal(out, want) and torch.isfinite(out.float()).all() and (counts >= 1).all()
print("fine")
'''
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]
