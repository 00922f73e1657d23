"""What is measured of the paged serving operators, and their plain forms.

Four operators of the serving path: rows of keys and values written into a
paged cache (rlt.paged_append), read back out of it (rlt.paged_read), a chunk
of new tokens attending over it (rlt.attend_paged), and drafted tokens
verified against the target's distribution (rlt.verify).

The cache: pages [n_pages][kv heads][2][page][head_dim] (keys, then values), a
table of page numbers per sequence, and for 8-bit caches e4m3 elements with
one power-of-two scale per block of 32 elements of a row (one exponent byte,
biased by 127). The chunk's rows are listed sequence after sequence
(cu_rows[n + 1]); the last of a sequence's rows is its position kv_len - 1.
"""
import math

import torch

own = False

BLOCK = 32          # elements of a row that share a scale
E4M3_MAX = 448.0
E_MIN = -110        # least exponent of a scale


# ------------------------------------------------------------------ the cases
def _write(name, n, rows_lo, rows_hi, kv_heads, dh, page, dtype, kind, pad=0):
    return dict(name=name, op="write", n=n, rows_lo=rows_lo, rows_hi=rows_hi, before=200,
                kv_heads=kv_heads, dh=dh, page=page, dtype=dtype, kind=kind, pad=pad)


def _read(name, n, rows_lo, rows_hi, kv_heads, dh, page, dtype, kind, pad=0):
    return dict(name=name, op="read", n=n, rows_lo=rows_lo, rows_hi=rows_hi, before=0,
                kv_heads=kv_heads, dh=dh, page=page, dtype=dtype, kind=kind, pad=pad)


def _attend(name, n, rows_lo, rows_hi, len_lo, len_hi, heads, kv_heads, dh, page, dtype, kind,
            window=0, lse=False, pad=0):
    return dict(name=name, op="attend", n=n, rows_lo=rows_lo, rows_hi=rows_hi, len_lo=len_lo,
                len_hi=len_hi, heads=heads, kv_heads=kv_heads, dh=dh, page=page, dtype=dtype,
                kind=kind, window=window, lse=lse, pad=pad)


def _verify(name, n, k, vocab, temperature, draft, ragged=False, position_major=False,
            masked=False):
    return dict(name=name, op="verify", n=n, k=k, vocab=vocab, temperature=temperature,
                draft=draft, ragged=ragged, position_major=position_major, masked=masked)


def listed():
    return [
        # one decoding step of the ~140M model's 64 slots: a row of each sequence, kept as it is
        _write("write_step_bf16", 64, 1, 1, 12, 64, 64, "bf16", "plain"),
        # prompts of 16 sequences of the tied model's shape stored in 8 bits
        _write("write_prompts_e4m3", 16, 700, 1300, 16, 128, 128, "bf16", "e4m3", pad=37),
        # one slot taken out of a cache of small pages, as a snapshot does
        _read("read_slot_bf16", 1, 777, 777, 12, 64, 16, "bf16", "plain"),
        # the prefixes of 32 sequences taken out of an 8-bit cache with shared heads
        _read("read_prefixes_e4m3", 32, 500, 4096, 8, 128, 64, "bf16", "e4m3"),
        # the smallest step: four sequences of the 50M model's shape, one token each
        _attend("attend_step_small", 4, 1, 1, 100, 1024, 8, 8, 64, 64, "bf16", "plain"),
        # a decoding step of 32 long sequences of the tied model's shape in 8 bits
        _attend("attend_step_e4m3", 32, 1, 1, 2000, 4096, 16, 16, 128, 128, "bf16", "e4m3"),
        # five tokens (four drafted) of each sequence, four query heads to a key head
        _attend("attend_drafts_gqa", 48, 5, 5, 1000, 8192, 32, 8, 128, 64, "bf16", "plain"),
        # a chunk of a long prompt behind 30 thousand positions
        _attend("attend_prompt_chunk", 1, 2048, 2048, 32768, 32768, 16, 16, 128, 128, "bf16",
                "plain"),
        # prompts and decoding steps in one batch, windowed, 8 bits, pages of 32
        _attend("attend_mixed_window", 40, 1, 512, 300, 4096, 12, 12, 64, 32, "bf16", "e4m3",
                window=1024, lse=True, pad=19),
        # short chunks in 32 bits
        _attend("attend_chunk_f32", 6, 1, 100, 100, 1024, 4, 4, 64, 16, "f32", "plain", lse=True),
        # two sequences, four drafted tokens, the framework's vocabulary
        _verify("verify_small", 2, 4, 32768, 1.0, True),
        # a full batch, drafts of unequal length, a large vocabulary, logits as the head writes
        # them position by position
        _verify("verify_batch", 64, 5, 131072, 0.8, True, ragged=True, position_major=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "attend", "verify"])
    page = rng.choice([16, 32, 48, 64, 128, 256])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    kind = rng.choice(["plain", "e4m3"])
    dh = rng.choice([32, 64, 64, 128, 128])
    kv_heads = rng.choice([1, 2, 3, 4, 8, 12, 16])
    if op in ("write", "read"):
        hi = _log(rng, 1, 2048)
        lo = rng.randint(1, hi)
        n = max(1, min(_log(rng, 1, 200), 16384 * 16 * 128 // (hi * kv_heads * dh)))
        make = _write if op == "write" else _read
        c = make("", n, lo, hi, kv_heads, dh, page, dtype, kind, pad=rng.choice([0, 0, 5]))
    elif op == "attend":
        group = rng.choice([1, 1, 2, 3, 4, 8])
        kv_heads = min(kv_heads, 32 // group)
        rows_hi = rng.choice([1, rng.randint(2, 16), _log(rng, 16, 1500)])
        rows_lo = rows_hi if rng.random() < 0.5 else rng.randint(1, rows_hi)
        len_hi = _log(rng, rows_hi, 32768)
        len_lo = rng.randint(max(1, len_hi // 4), len_hi)
        # within the listed cases: scores of the plain form, bytes of the cache in 32 bits
        most = min(2 ** 30 // (rows_hi * len_hi * kv_heads * group),
                   2 ** 29 // (len_hi * kv_heads * dh))
        if dtype == "f32":
            most //= 8
        n = max(1, min(_log(rng, 1, 200), most))
        if most < 1:
            rows_hi = rows_lo = max(1, min(rows_hi, 2 ** 27 // (len_hi * kv_heads * group)))
        window = rng.choice([0, 0, _log(rng, 16, 2048)])
        c = _attend("", n, rows_lo, rows_hi, len_lo, len_hi, kv_heads * group, kv_heads, dh, page,
                    dtype, kind, window, rng.random() < 0.5, rng.choice([0, 0, 7]))
    else:
        vocab = _log(rng, 300, 131072)
        k = rng.randint(1, 8)
        n = max(1, min(_log(rng, 1, 256), 64 * 5 * 131072 // (vocab * k)))
        c = _verify("", n, k, vocab, rng.choice([0.0, 0.6, 1.0, 1.3]),
                    rng.random() < 0.7, rng.random() < 0.5, rng.random() < 0.5,
                    rng.random() < 0.5)
    del c["name"]
    return c


def _spread(n, lo, hi, phase):
    """n whole numbers over lo..hi, the ends among them where n allows: the same for every seed."""
    v = [lo + int(((i + 1) * 0.6180339887 + phase) % 1.0 * (hi - lo + 1)) for i in range(n)]
    v[0] = hi
    if n > 1:
        v[-1] = lo
    return v


def _rows_and_lengths(c):
    if c["op"] == "attend":
        rows = _spread(c["n"], c["rows_lo"], c["rows_hi"], 0.1)
        lens = [max(a, b) for a, b in zip(rows, _spread(c["n"], c["len_lo"], c["len_hi"], 0.7))]
    else:
        rows = _spread(c["n"], c["rows_lo"], c["rows_hi"], 0.1)
        lens = [r + (c["before"] * (i % 3)) // 2 for i, r in enumerate(rows)]
    return rows, lens


def _draft_lengths(c):
    return _spread(c["n"], 0, c["k"], 0.3) if c["ragged"] else [c["k"]] * c["n"]


# ----------------------------------------------------------------- the inputs
def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if c["op"] == "verify":
        n, k, V = c["n"], c["k"], c["vocab"]
        shape = (k + 1, n, V) if c["position_major"] else (n, k + 1, V)
        target = randn(*shape).mul_(3.0)
        if c["masked"]:  # words that the request forbids
            target.masked_fill_(torch.rand(V, generator=g, device="cuda") < 0.02, -math.inf)
        if c["position_major"]:
            target = target.transpose(0, 1)
        # the draft model's own logits: near the target's
        noisy = (target[:, :k] + 0.7 * randn(n, k, V)).contiguous()
        pick = noisy if c["temperature"] == 0 else noisy / c["temperature"] - torch.log(
            -torch.log(torch.rand((n, k, V), generator=g, device="cuda").clamp_(1e-20, 1 - 1e-7)))
        tokens = pick.argmax(-1).to(torch.int32)
        uniforms = torch.rand((n, k + 1), generator=g, device="cuda")
        lens = torch.tensor(_draft_lengths(c), dtype=torch.int32, device="cuda")
        return dict(c=c, target=target, draft=noisy if c["draft"] else None, tokens=tokens,
                    uniforms=uniforms, lens=lens)

    rows, lens = _rows_and_lengths(c)
    n, P, H, dh = c["n"], c["page"], c["kv_heads"], c["dh"]
    need = [-(-L // P) for L in lens]
    n_pages, width = sum(need) + 3, max(need) + 1
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(n):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
    cu = [0]
    for r in rows:
        cu.append(cu[-1] + r)
    total = cu[-1] + c["pad"]
    dt = _dtype(c)
    # keys have a few strong entries, as projections do
    strong = torch.exp(0.5 * randn(1, H, 2, 1, dh))
    strong[:, :, 1] = 1.0
    pages = torch.empty((n_pages, H, 2, P, dh), dtype=torch.float32, device="cuda")
    for i in range(0, n_pages, 512):
        part = pages[i:i + 512]
        part.copy_(randn(*part.shape)).mul_(strong)
    s = dict(c=c, table=table, cu=torch.tensor(cu, dtype=torch.int32, device="cuda"),
             kv_len=torch.tensor(lens, dtype=torch.int32, device="cuda"), scales=None)
    if c["kind"] == "e4m3":
        s["pages"], s["scales"] = _quantise(pages)
    else:
        s["pages"] = pages.to(dt)
    if own:
        from token_recurrent_decoding_b200 import rlt
        s["cache"] = rlt.PagedKV(s["pages"], s["scales"], dtype=dt)
    if c["op"] == "attend":
        heads = c["heads"]
        # the queries are a part of the fused q | k | v projection's rows
        fused = randn(total, heads + 2 * H, dh).mul_(1.5).to(dt)
        s.update(q=fused[:, :heads], out=torch.zeros((total, heads, dh), dtype=dt, device="cuda"),
                 lse=torch.zeros((total, heads), device="cuda") if c["lse"] else None,
                 max_rows=max(rows), max_len=max(lens))
        if own:
            s["work"] = torch.empty(
                rlt.attend_paged_workspace_bytes(s["cache"], n, heads, total, max(rows), max(lens)),
                dtype=torch.uint8, device="cuda")
    else:
        fused = (randn(total, 2, H, dh) * strong[0, :, :, 0].transpose(0, 1)).to(dt)
        s.update(k=fused[:, 0], v=fused[:, 1],
                 k_out=torch.zeros((total, H, dh), dtype=dt, device="cuda"),
                 v_out=torch.zeros((total, H, dh), dtype=dt, device="cuda"))
    return s


# ------------------------------------------------------------ the plain forms
def _pow2(e):
    """2^e in 32 bits for whole e in -126..127, from its bits."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantise(x):
    """e4m3 elements and exponent bytes of x [..., dh] in 32 bits: per block the least power of
    two 2^e with |x| <= 448 * 2^e, and x * 2^-e (exact) rounded once. A block with an infinity
    or a NaN is stored as a whole as NaN: zeros under the exponent byte 255."""
    shape = x.shape
    x = x.reshape(*shape[:-1], -1, min(BLOCK, shape[-1]))
    fine = torch.isfinite(x).all(-1, keepdim=True)
    top = torch.where(fine, x, 0.0).abs().amax(-1, keepdim=True)
    mant, e = torch.frexp(top)                     # top = mant * 2^e, mant in [0.5, 1)
    e = e - 9 + (mant > E4M3_MAX / 512).to(e.dtype)
    e = torch.where(top > 0, e, E_MIN).clamp(min=E_MIN)
    y = torch.where(fine, x * _pow2(-e), 0.0)
    e = torch.where(fine, e, 128)
    return (y.to(torch.float8_e4m3fn).reshape(shape).contiguous(),
            (e + 127).squeeze(-1).to(torch.uint8).contiguous())


def _values(pages, scales):
    """What a cache's elements stand for, in 32 bits."""
    x = pages.float()
    if scales is None:
        return x
    shape = x.shape
    x = x.reshape(*shape[:-1], scales.shape[-1], -1)
    return (x * _pow2(scales.int() - 127).unsqueeze(-1)).reshape(shape)


def _row_places(s):
    """Of each listed row: its sequence, and its page and place in the page."""
    cu, P = s["cu"].long(), s["c"]["page"]
    row = torch.arange(s["k"].shape[0], device="cuda")
    row = row[row < cu[-1]]
    seq = torch.searchsorted(cu, row, right=True) - 1
    pos = s["kv_len"].long()[seq] - cu[seq + 1] + row
    return row, s["table"].long()[seq, pos // P], pos % P


def _plain_write(s):
    row, page, place = _row_places(s)
    x = torch.stack([s["k"][row], s["v"][row]], 2)                  # [rows][H][2][dh]
    if s["scales"] is None:
        s["pages"][page, :, :, place] = x
    else:
        y, e = _quantise(x.float())
        s["pages"].view(torch.uint8)[page, :, :, place] = y.view(torch.uint8)
        s["scales"][page, :, :, place] = e


def _plain_read(s):
    row, page, place = _row_places(s)
    x = s["pages"].view(torch.uint8)[page, :, :, place].view(torch.float8_e4m3fn) \
        if s["scales"] is not None else s["pages"][page, :, :, place]
    x = _values(x, None if s["scales"] is None else s["scales"][page, :, :, place])
    s["k_out"][row] = x[:, :, 0].to(s["k_out"].dtype)
    s["v_out"][row] = x[:, :, 1].to(s["v_out"].dtype)


def _plain_attend(s):
    c = s["c"]
    n, H, dh, P = c["n"], c["kv_heads"], c["dh"], c["page"]
    group, R, L = c["heads"] // H, s["max_rows"], s["max_len"]
    cu, lens = s["cu"].long(), s["kv_len"].long()
    m = cu[1:] - cu[:-1]
    # keys and values, dense: [n][H][L][dh]
    tab = s["table"].long()[:, :-(-L // P)].clamp(min=0)
    pages = s["pages"].view(torch.uint8)[tab].view(torch.float8_e4m3fn) \
        if s["scales"] is not None else s["pages"][tab]
    x = _values(pages, None if s["scales"] is None else s["scales"][tab])
    x = x.permute(3, 0, 2, 1, 4, 5).reshape(2, n, H, -1, dh)[:, :, :, :L]
    i, j = torch.arange(R, device="cuda"), torch.arange(L, device="cuda")
    src = (cu[:-1, None] + i).clamp(max=max(s["q"].shape[0] - 1, 0))        # [n][R]
    q = s["q"][src].float().reshape(n, R, H, group, dh).permute(0, 2, 3, 1, 4)
    scores = torch.matmul(q.reshape(n, H, group * R, dh) / math.sqrt(dh), x[0].transpose(-1, -2))
    pos = (lens - m)[:, None] + i                                            # [n][R]
    hidden = j[None, None] > pos[..., None]
    if c["window"]:
        hidden |= j[None, None] <= pos[..., None] - c["window"]
    scores = scores.reshape(n, H, group, R, L).masked_fill_(hidden[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, 0.0)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.reshape(n, H, group * R, L), x[1]).reshape(n, H, group, R, dh)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).reshape(n, R, H * group, dh)
    lse = (top + torch.log(total)).squeeze(-1).permute(0, 3, 1, 2).reshape(n, R, H * group)
    row = torch.arange(s["q"].shape[0], device="cuda")
    row = row[row < cu[-1]]
    seq = torch.searchsorted(cu, row, right=True) - 1
    s["out"][row] = o[seq, row - cu[seq]].to(s["out"].dtype)
    if s["lse"] is not None:
        s["lse"][row] = lse[seq, row - cu[seq]]


def _weights(logits, temperature):
    """Softmax weights in 64 bits, and their sum."""
    x = logits.double()
    w = torch.exp((x - x.amax(-1, keepdim=True)) / temperature)
    return w, w.sum(-1, keepdim=True)


def _plain_verify(s):
    c = s["c"]
    n, k, tau = c["n"], c["k"], c["temperature"]
    tok, lens, u = s["tokens"].long(), s["lens"].long(), s["uniforms"].double()
    place = torch.arange(k, device="cuda")
    if tau == 0:
        best = s["target"].argmax(-1)
        fine = tok == best[:, :k]
    else:
        wp, zp = _weights(s["target"], tau)
        px = wp[:, :k].gather(-1, tok[..., None]).squeeze(-1)
        if s["draft"] is not None:
            wq, zq = _weights(s["draft"], tau)
            qx = wq.gather(-1, tok[..., None]).squeeze(-1)
            fine = u[:, :k] * qx * zp[:, :k, 0] < px * zq[..., 0]
        else:
            fine = u[:, :k] * zp[:, :k, 0] < px
    fine &= place < lens[:, None]
    count = torch.cumprod(fine.long(), 1).sum(1)                              # accepted
    at = torch.arange(n, device="cuda")
    if tau == 0:
        new = best[at, count]
    else:
        w = wp[at, count] / zp[at, count]
        refused = (count < lens)[:, None]
        j = count.clamp(max=k - 1)
        if s["draft"] is not None:
            rest = (w - wq[at, j] / zq[at, j]).clamp(min=0)
        else:
            rest = w.scatter(1, tok[at, j][:, None], 0.0)
        w = torch.where(refused, rest, w)
        cum = w.cumsum(-1)
        new = (cum <= u[:, k:] * cum[:, -1:]).sum(-1)
        last = c["vocab"] - 1 - (w.flip(-1) > 0).int().argmax(-1)
        new = torch.minimum(new, last)
    out = torch.full((n, k + 1), -1, dtype=torch.int32, device="cuda")
    out[:, :k] = torch.where(place < count[:, None], s["tokens"], -1)
    out[at, count] = new.int()
    return out, (count + 1).int()


# -------------------------------------------------------------------- one pass
def run(s):
    c = s["c"]
    if own:
        from token_recurrent_decoding_b200 import rlt
    if c["op"] == "write":
        if own:
            rlt.paged_append(s["cache"], s["table"], s["k"], s["v"], s["cu"], s["kv_len"])
            rlt.paged_read(s["cache"], s["table"], s["cu"], s["kv_len"], s["k_out"], s["v_out"])
        else:
            _plain_write(s)
            _plain_read(s)
        return s["k_out"], s["v_out"]
    if c["op"] == "read":
        if own:
            rlt.paged_read(s["cache"], s["table"], s["cu"], s["kv_len"], s["k_out"], s["v_out"])
        else:
            _plain_read(s)
        return s["k_out"], s["v_out"]
    if c["op"] == "attend":
        if own:
            rlt.attend_paged(s["q"], s["cache"], s["table"], s["cu"], s["kv_len"], s["max_rows"],
                             s["max_len"], out=s["out"], lse=s["lse"], window=c["window"],
                             workspace=s["work"])
        else:
            _plain_attend(s)
        return [s["out"]] + ([s["lse"]] if c["lse"] else [])
    if own:
        return rlt.verify(s["target"], s["draft"], s["tokens"], c["temperature"], s["uniforms"],
                          draft_lengths=s["lens"])
    return _plain_verify(s)


# ------------------------------------------------- what a pass cannot do without
def work(c):
    if c["op"] == "verify":
        drafted = sum(_draft_lengths(c))
        rows = drafted + c["n"] + (drafted if c["draft"] and c["temperature"] else 0)
        return {"bytes": rows * c["vocab"] * 4.0, "flops": 4.0 * rows * c["vocab"]}
    rows, lens = _rows_and_lengths(c)
    es = 2 if c["dtype"] == "bf16" else 4
    H, dh = c["kv_heads"], c["dh"]
    cell = 2 * H * dh * (es if c["kind"] == "plain" else 1 + 1 / min(BLOCK, dh))
    if c["op"] != "attend":
        dense, kept = sum(rows) * 2 * H * dh * es, sum(rows) * cell
        # written rows are read back: dense in, cache out, cache in, dense out
        return {"bytes": float((dense + kept) * (2 if c["op"] == "write" else 1)),
                "flops": float(sum(rows) * 2 * H * dh)}
    W = c["window"] or 1 << 40
    pairs = keys = 0
    for m, L in zip(rows, lens):
        first = L - m
        keys += L - max(0, first - W + 1)
        short = min(m, max(0, W - first))            # rows whose window reaches the start
        pairs += (2 * first + 1 + short) * short // 2 + (m - short) * W
    q = sum(rows) * c["heads"] * dh * es
    return {"bytes": float(keys * cell + 2 * q), "flops": 4.0 * dh * c["heads"] * pairs}


# ------------------------------------------------------ the definition, 64 bits
def _e4m3_table():
    """The value of each of the 256 codes: sign, four exponent bits (bias 7), three of fraction."""
    v = []
    for code in range(256):
        e, f = code >> 3 & 15, code & 7
        x = f / 8 * 2.0 ** -6 if e == 0 else math.nan if code & 127 == 127 else \
            (1 + f / 8) * 2.0 ** (e - 7)
        v.append(-x if code >> 7 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _pow64(e):
    """2^e in 64 bits, from its bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _stored64(x):
    """What rows x [..., dh] stand for once stored in 8 bits."""
    shape, grid = x.shape, _e4m3_table()[:127]
    x = x.double().reshape(-1, min(BLOCK, shape[-1]))
    top = x.abs().amax(1, keepdim=True)
    e = torch.ceil(torch.log2(top / E4M3_MAX)).clamp(min=E_MIN)
    e = torch.where(top > E4M3_MAX * _pow64(e), e + 1, e)
    e = torch.where(top <= E4M3_MAX * _pow64(e - 1), e - 1, e).clamp(min=E_MIN)
    y = (x * _pow64(-e)).abs()
    hi = torch.searchsorted(grid, y).clamp(1, 126)
    below, above = grid[hi - 1], grid[hi]
    up = (y - below > above - y) | ((y - below == above - y) & (hi % 2 == 0))
    return (torch.where(up, above, below) * torch.sign(x) * _pow64(e)).reshape(shape)


def _held64(s, b):
    """Sequence b's keys and values [len][H][2][dh] as stored, page after page."""
    L, P = int(s["kv_len"][b]), s["c"]["page"]
    ids = s["table"][b, :-(-L // P)].long()
    x = s["pages"][ids] if s["scales"] is None else s["pages"].view(torch.uint8)[ids]
    if s["scales"] is not None:
        scale = _pow64(s["scales"][ids].long() - 127)
        x = _e4m3_table()[x.long()] * scale.repeat_interleave(x.shape[-1] // scale.shape[-1], -1)
    return x.double().permute(0, 3, 1, 2, 4).reshape(-1, x.shape[1], 2, x.shape[-1])[:L]


def _exact_attend(c, s):
    cu = s["cu"].tolist()
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(out.shape[:2], dtype=torch.float64, device="cuda")
    group = c["heads"] // c["kv_heads"]
    for b in range(c["n"]):
        kv = _held64(s, b)
        lo, hi, L = cu[b], cu[b + 1], kv.shape[0]
        pos = torch.arange(L - (hi - lo), L, device="cuda")[:, None]
        key = torch.arange(L, device="cuda")[None]
        seen = (key <= pos) & ((key > pos - c["window"]) if c["window"] else True)
        for h in range(c["heads"]):
            z = s["q"][lo:hi, h].double() @ kv[:, h // group, 0].T * c["dh"] ** -0.5
            z = torch.where(seen, z, -math.inf)
            out[lo:hi, h] = torch.softmax(z, -1) @ kv[:, h // group, 1]
            lse[lo:hi, h] = torch.logsumexp(z, -1)
    return [out] + ([lse] if c["lse"] else [])


def _exact_verify(c, s):
    n, k, tau, V = c["n"], c["k"], c["temperature"], c["vocab"]
    out, many = [], []
    lens, tok, u = s["lens"].tolist(), s["tokens"].tolist(), s["uniforms"].double()
    for b in range(n):
        got, j = [], 0
        while True:
            row = s["target"][b, j].double()
            if tau == 0:
                best = int((row == row.max()).int().argmax())
                got.append(best)
                if j < lens[b] and tok[b][j] == best:
                    j += 1
                    continue
                break
            p = torch.softmax(row / tau, 0)
            if j < lens[b]:
                x = tok[b][j]
                if s["draft"] is not None:
                    q = torch.softmax(s["draft"][b, j].double() / tau, 0)
                else:
                    q = torch.zeros(V, dtype=torch.float64, device="cuda")
                    q[x] = 1.0
                if bool(u[b, j] * q[x] < p[x]):
                    got.append(x)
                    j += 1
                    continue
                p = torch.relu(p - q)
            cum = torch.cumsum(p, 0)
            v = int(torch.searchsorted(cum, (u[b, k] * cum[-1]).reshape(1), right=True))
            got.append(min(v, int(torch.nonzero(p).max())))
            break
        many.append(len(got))
        out.append(got + [-1] * (k + 1 - len(got)))
    return (torch.tensor(out, dtype=torch.int32, device="cuda"),
            torch.tensor(many, dtype=torch.int32, device="cuda"))


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "attend":
        return _exact_attend(c, s)
    if c["op"] == "verify":
        return _exact_verify(c, s)
    cu = s["cu"].tolist()
    out = [torch.zeros(s["k_out"].shape, dtype=torch.float64, device="cuda") for _ in range(2)]
    for b in range(c["n"]):
        lo, hi = cu[b], cu[b + 1]
        if c["op"] == "read":
            kv = _held64(s, b)[-(hi - lo):]
            got = kv[:, :, 0], kv[:, :, 1]
        elif c["kind"] == "e4m3":
            got = _stored64(s["k"][lo:hi]), _stored64(s["v"][lo:hi])
        else:
            got = s["k"][lo:hi].double(), s["v"][lo:hi].double()
        out[0][lo:hi], out[1][lo:hi] = got
    return tuple(out)
