"""The paged cache and the attention over it where values stop being finite, at the ends of their
types and at the ends of the arguments' ranges: on the GPU, against float64 on the CPU."""
import math

import pytest
import torch

from paged_cases import BF16, F32, Case, attend64, attend_bound, quantised
from token_recurrent_decoding_b200 import rlt

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "f32", "bf16e4", "f32e4"]


def _case(kind, rows, lens, **kw):
    return Case(rows, lens, dtype=F32 if kind[0] == "f" else BF16, e4=kind.endswith("e4"), **kw)


def _place(c, b, pos):
    return int(c.table[b, pos // c.page]), pos % c.page


def _spoil(c, b, head, kv, pos, value):
    """The whole key or value of one position and head becomes `value` (8 bits: NaN)."""
    pg, sl = _place(c, b, pos)
    if c.e4:
        c.scales[pg, head, kv, sl] = 255
        c.pages.view(torch.uint8)[pg, head, kv, sl] = 0
    else:
        c.pages[pg, head, kv, sl] = value


def _sees(c, b, pos, window):
    """[m] whether row i of sequence b sees key `pos`."""
    p = c.lens[b] - c.rows[b] + torch.arange(c.rows[b])
    return (pos <= p) & ((pos > p - window) if window else torch.ones_like(p, dtype=torch.bool))


# (8 bits hold a NaN only: an infinity is stored as one)
@pytest.mark.parametrize("kind,value", [(k, math.nan) for k in KINDS] +
                         [("bf16", math.inf), ("f32", math.inf)])
@pytest.mark.parametrize("m,before,group,dh,window", [
    (256, 0, 1, 64, 0), (256, 0, 1, 128, 0), (300, 37, 1, 64, 0), (130, 0, 2, 128, 0),
    (150, 21, 3, 64, 0), (300, 0, 1, 64, 140), (256, 200, 2, 64, 90), (257, 5, 1, 128, 128)])
def test_rows_that_see_a_value_that_is_not_finite(kind, value, m, before, group, dh, window):
    """Wherever it lies among the tiles and whichever other rows see it: those rows are not finite
    (NaN from a NaN), all others are as without it."""
    L = m + before
    c = _case(kind, [m], [L], H=2, dh=dh, page=32, seed=m + group).device()
    q = c.queries(2 * group)
    dq = q.cuda()
    clean = c.pages.clone(), None if c.scales is None else c.scales.clone()
    held, seen = c.kv[0].clone(), 0
    for pos in (5, 100, 127, 128, 200, L - 2):
        if pos >= L:
            continue
        c.pages.copy_(clean[0])
        if c.e4:
            c.scales.copy_(clean[1])
        _spoil(c, 0, 1, 1, pos, value)
        c.device()
        c.kv[0] = held.clone()
        c.kv[0][pos, 1, 1] = 0.0
        lse = torch.zeros((m, 2 * group), device="cuda")
        out = rlt.attend_paged(dq, c.cache, c.d_table, c.d_cu, c.d_len, m, L, lse=lse,
                               window=window).double().cpu()
        ref, _, mass, size = attend64(q.double(), c.kv[0], L, window)
        hit = torch.zeros((m, 2 * group), dtype=torch.bool)
        hit[:, group:] = _sees(c, 0, pos, window)[:, None]
        seen += int(hit.any())
        assert not torch.isfinite(out[hit]).any(), pos
        if value != value:
            assert torch.isnan(out[hit]).all(), pos
        bound = attend_bound(ref, mass, size, dh, c.dtype)
        assert ((out - ref).abs()[~hit] <= bound[~hit]).all(), pos
        assert torch.isfinite(lse.cpu()[~hit]).all(), pos
    assert seen > 0


# ------------------------------------------------------------------ other streams
def _pool_of(t):
    """The stream whose memory t lies in."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the allocator's")


def _calls(c, side):
    """The calls that make their own buffers, on `side`, with what they give on the current stream."""
    q = c.queries(4).cuda()
    t = torch.randn((64, 3, 5000), device="cuda")
    x = torch.zeros((64, 2), dtype=torch.int32, device="cuda")
    u = torch.full((64, 3), 0.5, device="cuda")
    attend = lambda s: (rlt.attend_paged(q, c.cache, c.d_table, c.d_cu, c.d_len, 40,  # noqa: E731
                                         3000, stream=s),)
    verify = lambda s: rlt.verify(t, t[:, :2], x, 1.0, u, stream=s)  # noqa: E731
    wants = [f(None) for f in (attend, verify)]
    torch.cuda.synchronize()
    return [(lambda: attend(side), wants[0]), (lambda: verify(side), wants[1])]


def test_buffers_of_a_call_on_another_stream_are_that_streams_own():
    c = _case("bf16", [1, 40], [3000, 900], H=2, dh=64, page=64, seed=1).device()
    side = torch.cuda.Stream()
    for call, want in _calls(c, side):
        got = call()
        assert all(_pool_of(t) == side.cuda_stream for t in got)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    # on the current stream, named or not, nothing changes
    here = torch.cuda.current_stream()
    for stream in (None, here):
        for call, _ in _calls(c, stream):
            assert all(_pool_of(t) == here.cuda_stream for t in call())


def test_a_call_on_another_stream_leaves_pending_work_alone():
    """Work of the current stream is still to read blocks that were freed behind it, of every size
    the calls may want, while they run on another stream."""
    c = _case("bf16", [1, 40], [3000, 900], H=2, dh=64, page=64, seed=1).device()
    side = torch.cuda.Stream()
    a = torch.randn((4096, 4096), device="cuda")
    for call, want in _calls(c, side):
        sizes = [2 ** i for i in range(9, 25)]
        kept = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda.synchronize()
        blocks = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda.synchronize()
        for _ in range(20):
            a @ a  # a few milliseconds
        for to, block in zip(kept, blocks):
            to.copy_(block)
        del blocks, block
        got = call()
        torch.cuda.synchronize()
        assert all((to == 7).all() for to in kept)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


# -------------------------------------------------------- the ends of the types
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("m", [3, 150])
@pytest.mark.parametrize("window", [0, 20])
@pytest.mark.parametrize("sign", [1, -1])
def test_the_largest_numbers_in_unseen_places_do_not_matter(kind, m, window, sign):
    """Keys and values of the type's largest or lowest value that only the last row sees."""
    L = m + 30
    c = _case(kind, [m], [L], H=1, dh=64, page=16, seed=3)
    for kv in (0, 1):
        _spoil(c, 0, 0, kv, L - 1, sign * torch.finfo(c.dtype).max)
    c.device()
    q = c.queries(2)
    out = rlt.attend_paged(q.cuda(), c.cache, c.d_table, c.d_cu, c.d_len, m, L,
                           window=window).double().cpu()
    ref, _, mass, size = attend64(q.double(), c.kv[0], L, window)
    assert ((out - ref).abs() <= attend_bound(ref, mass, size, 64, c.dtype))[:-1].all()


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("dh", [16, 32, 64, 128])
def test_the_largest_numbers_are_values_like_others(kind, dh):
    """One key: its weight is one, so its value comes out, to the two roundings of the division."""
    c = _case(kind, [1], [1], H=1, dh=dh, page=16, seed=3)
    top = torch.finfo(c.dtype).max
    c.pages[:, :, 1] = top
    c.pages[:, :, 1, :, ::2] = -top
    c.device()
    q = c.queries(1)
    out = rlt.attend_paged(q.cuda(), c.cache, c.d_table, c.d_cu, c.d_len, 1, 1).double().cpu()
    want = torch.full((dh,), top, dtype=torch.float64)
    want[::2] = -top
    assert ((out[0, 0] - want).abs() <= 2.0 ** -23 * top).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m", [2, 40, 150])
@pytest.mark.parametrize("size", [1e4, 1e9, 1e13, 1e36])
def test_scores_far_beyond_the_exponent(kind, m, size):
    """Scores of up to 1e36, finite in fp32: one key takes nearly every row, whatever the spacing of
    fp32 there is (the scores are single products, so that no order of a sum decides)."""
    L, dh = m + 70, 64
    c = _case(kind, [m], [L], H=1, dh=dh, page=16, seed=4).device()
    q = c.queries(2) * math.sqrt(size)
    q[:, :, 1:] = 0
    if not c.e4:
        c.d_pages[:, :, 0] *= math.sqrt(size)
        c.kv[0][:, :, 0] = (c.kv[0][:, :, 0].to(c.dtype).cuda() * math.sqrt(size)).double().cpu()
    lse = torch.zeros((m, 2), device="cuda")
    out = rlt.attend_paged(q.cuda(), c.cache, c.d_table, c.d_cu, c.d_len, m, L,
                           lse=lse).double().cpu()
    ref, rl, mass, size = attend64(q.double(), c.kv[0], L, 0)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    # a score's own roundings, as attend_bound counts them, and where they leave the winner open
    # (another key within them), any mean of values
    bound = attend_bound(ref, mass, size, dh, c.dtype)
    top = c.kv[0][:, 0, 1].abs().max() * 2
    assert ((out - ref).abs() <= bound.clamp(max=top)).all()
    lb = size * (dh + 8) * 2.0 ** -23 + 512 * 2.0 ** -23 + rl.abs() * 2.0 ** -22
    assert ((lse.double().cpu() - rl).abs() <= lb).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("dh", [16, 64])
@pytest.mark.parametrize("m", [3, 150])
def test_the_largest_numbers_in_8_bits(dtype, dh, m):
    """What is written from finite numbers reads back finite: from 248 * 2^120 on, where the nearest
    element would be 2^128, as 240 * 2^120. Rows that do not see them are as without them."""
    L, top = m + 30, torch.finfo(dtype).max
    c = Case([m], [L], H=2, dh=dh, page=16, seed=3, dtype=dtype, e4=True)
    x = torch.randn((m, 4, dh), generator=c.g).to(dtype)
    edges = torch.tensor([top, -top, 248 * 2.0 ** 120, -249 * 2.0 ** 120, 240 * 2.0 ** 120,
                          247 * 2.0 ** 120, 2.0 ** 127, 1.0], dtype=torch.float64).to(dtype)
    x[-1, :, :] = edges.repeat(dh // 8)
    x[0, 0] = 447 * 2.0 ** 119  # the first head's key, under the scale below: 448 * 2^119
    c.device()
    dx = x.cuda()
    rlt.paged_append(c.cache, c.d_table, dx[:, :2], dx[:, 2:], c.d_cu, c.d_len)
    ko, vo = (torch.empty((m, 2, dh), dtype=dtype, device="cuda") for _ in range(2))
    rlt.paged_read(c.cache, c.d_table, c.d_cu, c.d_len, ko, vo)
    want = torch.from_numpy(quantised(x.double().numpy())[0])
    assert (want.abs() >= 2.0 ** 128).any()
    want = want.clamp(-240 * 2.0 ** 120, 240 * 2.0 ** 120)
    got = torch.cat([ko, vo], 1).double().cpu()
    assert torch.isfinite(got).all() and torch.equal(got, want)
    held = c.kv[0].clone()
    held[L - m:] = torch.stack([want[:, :2], want[:, 2:]], 2)
    q = c.queries(2) / 64
    q[:, :, 1:] = 0  # scores of the largest keys stay finite
    out = rlt.attend_paged(q.cuda(), c.cache, c.d_table, c.d_cu, c.d_len, m, L).double().cpu()
    ref, _, mass, size = attend64(q[1:].double(), held, L, 0)
    assert torch.isfinite(out[:-1]).all()
    ok = attend_bound(ref, mass, size, dh, dtype)
    assert ((out[1:-1, 1] - ref[:-1, 1]).abs() <= ok[:-1, 1]).all()


# ------------------------------------------------- the ends of the arguments' ranges
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m", [5, 100])
def test_the_largest_windows_hide_nothing(kind, m):
    """Also where the first rows lie before position 0."""
    c = _case(kind, [m], [m], H=1, dh=64, page=16, seed=3).device()
    q = c.queries(2).cuda()
    short = c.d_len - 3
    want = rlt.attend_paged(q, c.cache, c.d_table, c.d_cu, short, m, m)
    assert (want[:3] == 0).all() and (want[3:] != 0).any()
    for window in (m - 3, m, m + 1, 2 ** 31 - 1):
        got = rlt.attend_paged(q, c.cache, c.d_table, c.d_cu, short, m, m, window=window)
        assert torch.equal(got, want), window


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_one_row_of_any_stride(kind):
    """A single row has no stride to speak of: q, k, v and out of odd or different ones."""
    c = _case(kind, [1], [40], H=2, dh=64, page=16, seed=2).device()
    want = rlt.attend_paged(c.queries(2).cuda(), c.cache, c.d_table, c.d_cu, c.d_len, 1, 40)
    c2 = _case(kind, [1], [40], H=2, dh=64, page=16, seed=2).device()

    def odd(x, more):
        flat = torch.zeros((1, 128 + more), dtype=c.dtype, device="cuda")
        flat[:, :128] = x.reshape(1, 128)
        y = flat.as_strided((1, 2, 64), (128 + more, 64, 1))
        assert y.stride(0) == 128 + more
        return y

    q = odd(c2.queries(2).cuda(), 3)
    out = odd(torch.zeros(128, device="cuda"), 5)
    rlt.attend_paged(q, c2.cache, c2.d_table, c2.d_cu, c2.d_len, 1, 40, out=out)
    assert torch.equal(out, want)
    k, v = (torch.randn((1, 2, 64), device="cuda").to(c.dtype) for _ in range(2))
    rlt.paged_append(c2.cache, c2.d_table, k, odd(v, 7), c2.d_cu, c2.d_len)
    ko, vo = odd(torch.zeros(128, device="cuda"), 1), torch.zeros_like(v)
    rlt.paged_read(c2.cache, c2.d_table, c2.d_cu, c2.d_len, ko, vo)
    assert torch.equal(ko, k) and torch.equal(vo, v)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dh,heads,H", [(16, 6, 3), (32, 2, 2), (64, 4, 2), (128, 3, 1)])
def test_queries_that_are_parts_of_wider_rows(kind, dh, heads, H):
    """q as a fused projection leaves it, on the GPU: row strides of q and out that are neither the
    rows' own size nor each other's, from steps to chunks of every kernel."""
    c = _case(kind, [1, 5, 150, 0, 40], [300, 64, 200, 9, 41], H=H, dh=dh, page=16, seed=dh,
              pad=3).device()
    wide = torch.randn((c.total, heads + 2 * H, dh), generator=c.g).to(c.dtype).cuda()
    q = wide[:, H:H + heads]
    out = torch.full((c.total, heads + 5, dh), 9.0, dtype=c.dtype, device="cuda")
    assert heads * dh < q.stride(0) != out.stride(0) > heads * dh
    rlt.attend_paged(q, c.cache, c.d_table, c.d_cu, c.d_len, 150, 300, out=out[:, 2:heads + 2])
    got, q = out.double().cpu(), q.double().cpu()
    assert (got[:, :2] == 9).all() and (got[:, heads + 2:] == 9).all()
    assert (got[int(c.cu[-1]):] == 9).all()
    for b, m in enumerate(c.rows):
        lo = int(c.cu[b])
        ref, _, mass, size = attend64(q[lo:lo + m], c.kv[b], c.lens[b], 0)
        err = (got[lo:lo + m, 2:heads + 2] - ref).abs()
        assert (err <= attend_bound(ref, mass, size, dh, c.dtype)).all(), b


# ------------------------------------------------------------- calls at their ends
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,m", [(40, 1), (128, 1), (129, 2), (1024, 1), (64, 5)])
def test_many_queries_share_one_key_head(kind, heads, m):
    """One token's heads alone fill the tiles of the many-row kernel."""
    c = _case(kind, [m, 1, 0], [700, 33, 5], H=1, dh=64, page=64, seed=heads).device()
    q = c.queries(heads)
    out = rlt.attend_paged(q.cuda(), c.cache, c.d_table, c.d_cu, c.d_len, m, 700).double().cpu()
    for b, lo in ((0, 0), (1, m)):
        ref, _, mass, size = attend64(q[lo:lo + c.rows[b]].double(), c.kv[b], c.lens[b], 0)
        err = (out[lo:lo + c.rows[b]] - ref).abs()
        assert (err <= attend_bound(ref, mass, size, 64, c.dtype)).all()


@pytest.mark.parametrize("kind", ["bf16", "f32", "bf16e4"])
@pytest.mark.parametrize("m", [1, 40])
def test_a_million_positions_on_a_few_pages(kind, m):
    """Positions past 2^20, every page in the table many times over."""
    page, L = 1024, 1_000_003
    c = _case(kind, [m], [16 * page], H=1, dh=64, page=page, seed=m).device()
    times = -(-L // page)
    table = c.d_table[:, :16].repeat(1, -(-times // 16))[:, :times].contiguous()
    kv = c.kv[0].repeat(times // 16 + 1, 1, 1, 1)[:L]
    q = c.queries(1)
    n = torch.tensor([L], dtype=torch.int32, device="cuda")
    out = rlt.attend_paged(q.cuda(), c.cache, table, c.d_cu, n, m, L).double().cpu()
    rows = [0] if m == 1 else [0, 17, m - 1]
    for i in rows:
        last = L - m + i + 1
        ref, _, mass, size = attend64(q[i:i + 1].double(), kv[:last], last, 0)
        # a lane adds up to 2 * L / 4096 terms one after the other instead of 512
        bound = attend_bound(ref, mass, size, 64, c.dtype) + mass * 2.0 ** -23 * L / 2048
        assert ((out[i:i + 1] - ref).abs() <= bound).all()


@pytest.mark.parametrize("kind", KINDS)
def test_the_output_may_take_the_queries_place(kind):
    c = _case(kind, [1, 5, 300, 40], [3000, 64, 400, 9000], H=2, dh=64, page=32, seed=6).device()
    q = c.queries(4).cuda()
    want = rlt.attend_paged(q, c.cache, c.d_table, c.d_cu, c.d_len, 300, 9000)
    got = rlt.attend_paged(q, c.cache, c.d_table, c.d_cu, c.d_len, 300, 9000, out=q)
    assert got.data_ptr() == q.data_ptr() and torch.equal(got, want)


@pytest.mark.parametrize("kind", [rlt.KV_PLAIN, rlt.KV_E4M3])
@pytest.mark.parametrize("H,dh,rows", [(1024, 16, 3), (300, 128, 40), (1, 16, 70000)])
def test_rows_of_many_heads_and_many_rows(kind, H, dh, rows):
    page = 1024
    pages = -(-rows // page)
    cache = rlt.PagedKV.empty(pages, page, H, dh, BF16, kind)
    g = torch.Generator(device="cuda").manual_seed(H)
    k, v = (torch.randn((rows, H, dh), generator=g, device="cuda").to(BF16) for _ in range(2))
    if kind == rlt.KV_E4M3:  # numbers that 8 bits hold: whole, of three bits
        k, v = (x.float().mul(2).round().clamp(-7, 7).to(BF16) for x in (k, v))
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.arange(pages, device="cuda").int().flip(0)[None].contiguous()
    rlt.paged_append(cache, table, k, v, i32(0, rows), i32(rows))
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    rlt.paged_read(cache, table, i32(0, rows), i32(rows), ko, vo)
    assert torch.equal(ko, k) and torch.equal(vo, v)


def test_a_captured_call_on_a_stream_forked_inside_the_capture():
    """Calls that make their own buffers, on another stream that joined the capture."""
    c = _case("bf16", [1, 40], [3000, 900], H=2, dh=64, page=64, seed=1).device()
    side = torch.cuda.Stream()
    calls = _calls(c, side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        gots = [call() for call, _ in calls]
        here.wait_stream(side)
    for _ in range(3):
        for got in gots:
            for t in got:
                t.zero_()
        graph.replay()
    torch.cuda.synchronize()
    for got, (_, want) in zip(gots, calls):
        assert all(torch.equal(a, b) for a, b in zip(got, want))
