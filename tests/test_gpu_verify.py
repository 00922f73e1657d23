"""Draft verification on the GPU against float64 on the CPU, and the paged operators together as a
speculative decoding loop."""
import math

import numpy as np
import pytest
import torch

from paged_cases import verify64
from token_recurrent_decoding_b200 import rlt

pytestmark = pytest.mark.gpu


def _run(target, draft, tokens, tau, u, lens=None, position_major=False):
    put = lambda x: None if x is None else (  # noqa: E731
        x.transpose(0, 1).contiguous().cuda().transpose(0, 1) if position_major else x.cuda())
    out, counts = rlt.verify(put(target), put(draft), tokens.int().cuda() if tokens is not None
                             else None, tau, None if u is None else u.cuda(),
                             draft_lengths=None if lens is None else
                             torch.tensor(lens, dtype=torch.int32).cuda())
    return out.cpu().numpy(), counts.cpu().numpy()


def _compare(target, draft, tokens, tau, u, lens=None, digits=0, **kw):
    n, k = target.shape[0], target.shape[1] - 1
    got = _run(target, draft, tokens, tau, u, lens, **kw)
    ref = verify64(target.double().numpy(), None if draft is None else draft.double().numpy(),
                   tokens.numpy() if k else np.zeros((n, 0), np.int64),
                   lens if lens is not None else [k] * n,
                   np.zeros((n, k + 1)) if u is None else u.double().numpy(), tau,
                   digits)
    # weights of 64 bits, sums of at most 2^17 of them: 2^-52 * 2^17 at the very worst
    assert ref[2] > 2.0 ** -35, "a comparison of this case is too near its border to be decided"
    assert np.array_equal(got[1], ref[1]), (got[1], ref[1])
    assert np.array_equal(got[0], ref[0])


def _inputs(n, k, V, seed, spread=3.0):
    g = torch.Generator().manual_seed(seed)
    target = torch.randn((n, k + 1, V), generator=g) * spread
    draft = target[:, :k] + 0.7 * torch.randn((n, k, V), generator=g)
    p = torch.softmax(draft, -1).reshape(-1, V)
    tokens = (torch.multinomial(p, 1, generator=g).reshape(n, k) if k else
              torch.zeros((n, 0), dtype=torch.long))
    return target, draft, tokens, torch.rand((n, k + 1), generator=g)


@pytest.mark.parametrize("tau", [0.0, 0.7, 1.0, 2.5])
@pytest.mark.parametrize("n,k,V", [(1, 0, 5), (3, 1, 1), (2, 4, 31), (5, 3, 4096), (4, 8, 4097),
                                   (7, 2, 33000), (1, 32, 300)])
def test_verification(tau, n, k, V):
    t, d, x, u = _inputs(n, k, V, seed=n + k + V)
    _compare(t, d, x, tau, u)
    _compare(t, None, x, tau, u, position_major=True)
    lens = [(3 * i) % (k + 2) - (i % 2) for i in range(n)]  # -1 .. k + 1: clamped
    _compare(t, d, x, tau, u, lens, position_major=True)


def test_large_vocabulary():
    t, d, x, u = _inputs(3, 2, 131072 + 5, seed=1)
    _compare(t, d, x, 0.9, u)


def test_forbidden_words_and_strange_logits():
    t, d, x, u = _inputs(6, 2, 500, seed=2)
    t[:, :, 100:400] = -math.inf
    d[0, :, 100:400] = -math.inf
    t[1, 0, 7] = math.nan          # no weight
    x[1, 0] = 7
    t[2, 0, 3] = t[2, 0, 9] = math.inf  # these two share the weight
    d[3] = -math.inf               # a draft without any weight
    t[4, 1] = -math.inf            # a target row without any weight
    x[5, 0] = 200                  # drafted although forbidden
    for tau in (0.0, 1.0):
        _compare(t, d, x, tau, u)
        _compare(t, None, x, tau, u)


def test_the_first_row_without_weight_has_no_token():
    t = torch.full((2, 2, 40), -math.inf)
    t[1, 1] = math.nan
    t[1, 0, 5] = 0.0
    x = torch.tensor([[3], [5]])
    u = torch.full((2, 2), 0.25)
    for tau in (0.0, 1.0):
        out, counts = _run(t, t[:, :1], x, tau, u)
        assert out.tolist() == [[-1, -1], [5, -1]] and counts.tolist() == [0, 1]


def test_tokens_outside_the_vocabulary_end_the_draft():
    t, d, x, u = _inputs(4, 3, 64, seed=3)
    x[0, 0], x[1, 1], x[2, 2] = -1, 64, 1 << 30
    for tau in (0.0, 1.0):
        _compare(t, d, x, tau, u)


def test_equal_maxima_and_uniform_ends():
    t = torch.zeros((2, 2, 37))
    x = torch.tensor([[0], [1]])
    out, counts = _run(t, None, x, 0.0, None)
    assert out.tolist() == [[0, 0], [0, -1]] and counts.tolist() == [2, 1]
    u = torch.tensor([[0.0, 0.0], [1 - 2.0 ** -24, 1 - 2.0 ** -24]])
    out, counts = _run(t, None, x, 1.0, u)
    # 0 < 1/37 accepted, then the first word; the other refused, then the last word
    assert out.tolist() == [[0, 0], [36, -1]] and counts.tolist() == [2, 1]


def test_huge_logits():
    t, d, x, u = _inputs(3, 2, 700, seed=4, spread=1e4)
    _compare(t, d, x, 1.0, u)
    t = t * 1e30
    x[:, 0] = t[:, 0].argmax(-1)
    _compare(t, t[:, :2].contiguous(), x, 0.5, u)


def test_nearly_equal_distributions():
    """p and q equal to 1e-6, with drafted words of no weight under p: refusals whose difference is
    tiny everywhere; and many words of equal weights in both."""
    t, _, x, u = _inputs(6, 2, 3000, seed=10)
    g = torch.Generator().manual_seed(3)
    d = t[:, :2] + 1e-6 * torch.randn(t[:, :2].shape, generator=g)
    for b in range(6):
        t[b, 0, x[b, 0]] = -math.inf
    _compare(t, d, x, 1.0, u)
    t, d, x, u = _inputs(6, 2, 3000, seed=11)
    t[:, :, ::2] = 1.0
    d[:, :, ::2] = 1.0
    _compare(t, d, x, 1.0, u)


@pytest.mark.parametrize("tau", [1e-3, 1e-40, 50.0])
def test_extreme_temperatures(tau):
    """At 1e-3 a row's p and q are both 1 - 1e-38 or so at one word: its difference, 1.7e-38 in one of
    these rows, is the draw's whole weight but not in 64 bits, so the reference takes decimals."""
    t, d, x, u = _inputs(5, 3, 900, seed=12)
    _compare(t, d, x, float(torch.tensor(tau, dtype=torch.float32)), u,
             digits=60 if tau == 1e-3 else 0)


def test_equal_distributions_accept_everything():
    t, _, x, u = _inputs(50, 4, 999, seed=5)
    out, counts = _run(t, t[:, :4].contiguous(), x, 1.0, u)
    assert (counts == 5).all() and np.array_equal(out[:, :4], x.numpy())


@pytest.mark.parametrize("with_draft", [True, False])
def test_close_tests_are_decided_exactly(with_draft):
    """Uniforms within 1e-6 of p / q on either side: closer than sums in 32 bits decide. With one
    drafted token after another of that kind, accepted and refused."""
    n, k, V = 24, 4, 20000
    t, d, x, u = _inputs(n, k, V, seed=9)
    p = torch.softmax(t[:, :k].double(), -1).gather(2, x[..., None])[..., 0]
    q = torch.softmax(d.double(), -1).gather(2, x[..., None])[..., 0] if with_draft else 1.0
    side = torch.tensor([[1 - 1e-6 if (b >> i) & 1 else 1 + 1e-6 for i in range(k)]
                         for b in range(n)], dtype=torch.float64)
    u[:, :k] = (p / q * side).float().clamp(max=0.9999)
    _compare(t, d if with_draft else None, x, 1.0, u)


def test_emitted_tokens_follow_the_target():
    """The first emitted token of many sequences with one distribution: its counts against n p.
    Each count is binomial; six of its standard deviations, and one, bound all 12 with a chance of
    error below 1e-7."""
    n, V = 60000, 12
    g = torch.Generator().manual_seed(6)
    t1, d1 = torch.randn(V, generator=g), torch.randn(V, generator=g)
    p, q = torch.softmax(t1.double(), 0), torch.softmax(d1.double(), 0)
    x = torch.multinomial(q, n, replacement=True, generator=g).reshape(n, 1)
    u = torch.rand((n, 2), generator=g)
    out, _ = _run(t1.expand(n, 2, V), d1.expand(n, 1, V).contiguous(), x, 1.0, u)
    counts = np.bincount(out[:, 0], minlength=V)
    sd = np.sqrt(n * p.numpy() * (1 - p.numpy()))
    assert (np.abs(counts - n * p.numpy()) <= 6 * sd + 1).all()


def test_captured_and_at_once():
    t, d, x, u = (a.cuda() for a in _inputs(9, 3, 5000, seed=7))
    x = x.int()
    want = rlt.verify(t, d, x, 1.0, u)
    work = torch.empty(rlt.verify_workspace_bytes(9, 3, 5000), dtype=torch.uint8, device="cuda")
    outs = [[torch.empty_like(w) for w in want] for _ in range(2)]
    graphs = []
    for o in outs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            rlt.verify(t, d, x, 1.0, u, tokens=o[0], counts=o[1], workspace=work)
        graphs.append(graph)
    for _ in range(3):
        for graph in graphs:
            graph.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o[0], want[0]) and torch.equal(o[1], want[1])
    streams = [torch.cuda.Stream() for _ in range(3)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    many = [rlt.verify(t, d, x, 1.0, u, stream=s) for _ in range(5) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(a, want[0]) and torch.equal(b, want[1]) for a, b in many)


def test_tensors_that_do_not_fit_are_refused():
    t, d, x, u = (a.cuda() for a in _inputs(2, 3, 50, seed=8))
    x = x.int()
    for args in ((t.double(), d, x, 1.0, u), (t, d[:, :2], x, 1.0, u), (t, d, x.long(), 1.0, u),
                 (t, d, x, 1.0, None), (t, d, x, -1.0, u), (t, d, x, math.nan, u),
                 (t.cpu(), d, x, 1.0, u), (t, d.cpu(), x, 1.0, u), (t[..., ::2], None, x, 1.0, u),
                 (t, d, None, 1.0, u), (t, d, x, 1.0, u[:, :3])):
        with pytest.raises(rlt.RLTError):
            rlt.verify(*args)
    with pytest.raises(rlt.RLTError):
        rlt.verify(t, d, x, 1.0, u, workspace=torch.empty(1, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------- the operators as they are used
class _Toy:
    """One attention layer with a head over the words: token -> q, k, v rows by lookup, the logits
    from the attention's output and the token itself. The projections are sums in float64, so a
    row's logits do not depend on how many rows are computed together."""

    def __init__(self, V, heads, H, dh, seed):
        g = torch.Generator().manual_seed(seed)
        self.qkv = torch.randn((V, heads + 2 * H, dh), generator=g).to(torch.bfloat16).cuda()
        self.head = torch.randn((heads * dh, V), generator=g).double().cuda()
        self.skip = torch.randn((V, V), generator=g).double().cuda()
        self.heads, self.H, self.dh, self.V = heads, H, dh, V

    def logits(self, cache, table, tokens, cu, kv_len, max_rows, max_len):
        x = self.qkv[tokens.long()]
        q, k, v = x.split([self.heads, self.H, self.H], 1)
        rlt.paged_append(cache, table, k, v, cu, kv_len)
        a = rlt.attend_paged(q, cache, table, cu, kv_len, max_rows, max_len)
        y = (a.double().flatten(1).unsqueeze(-1) * self.head).sum(1)
        return (2.0 * y + self.skip[tokens.long()]).float()


@pytest.mark.parametrize("kind", [rlt.KV_PLAIN, rlt.KV_E4M3])
def test_speculative_decoding_emits_what_plain_decoding_does(kind):
    """Three sequences of one model: greedy, one token at a time, against drafts of four verified
    in one chunk, refused rows overwritten by the next chunk. Drafts are the right words with some
    mistakes. A row's result does not depend on its chunk, so the tokens are equal."""
    V, n, k, steps, page = 61, 3, 4, 40, 16
    toy = _Toy(V, 4, 2, 64, seed=3)
    prompts = [[1, 2, 3, 4, 5], [7], [9, 8, 7, 6, 5, 4, 3, 2, 1, 0, 9, 8, 7, 6, 5, 4, 3]]
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def start():
        cache = rlt.PagedKV.empty(n * 8, page, 2, 64, torch.bfloat16, kind)
        table = torch.randperm(n * 8, generator=torch.Generator().manual_seed(2)).int()
        table = table.reshape(n, 8).cuda()
        cu = [0]
        for p in prompts:
            cu.append(cu[-1] + len(p))
        flat = i32([t for p in prompts for t in p])
        logits = toy.logits(cache, table, flat, i32(cu), i32([len(p) for p in prompts]), 17, 17)
        return cache, table, logits[i32(cu[1:]).long() - 1].argmax(-1).int()

    cache, table, last = start()
    plain = [[int(t)] for t in last]
    lens = [len(p) for p in prompts]
    for _ in range(steps):
        lens = [x + 1 for x in lens]
        out = toy.logits(cache, table, i32([s[-1] for s in plain]), i32([0, 1, 2, 3]), i32(lens),
                         1, 100)
        for s, t in zip(plain, rlt.verify(out[:, None], None, None, 0.0)[0][:, 0].tolist()):
            s.append(t)

    cache, table, last = start()
    spec = [[int(t)] for t in last]
    lens = [len(p) for p in prompts]
    rounds = accepted = 0
    while min(len(s) for s in spec) <= steps:
        drafts = []
        for b, s in enumerate(spec):
            right = plain[b][len(s):len(s) + k] + [0] * k
            drafts.append([(t + (1 if (rounds + i + b) % 4 == 3 else 0)) % V
                           for i, t in enumerate(right[:k])])
        chunk = [[s[-1]] + d for s, d in zip(spec, drafts)]
        out = toy.logits(cache, table, i32([t for c in chunk for t in c]),
                         i32([0, 5, 10, 15]), i32([x + k + 1 for x in lens]), 5, 100)
        toks, counts = rlt.verify(out.view(n, k + 1, V), None, i32(drafts), 0.0)
        for b in range(n):
            c = int(counts[b])
            spec[b] += toks[b, :c].tolist()
            lens[b] += c
            accepted += c - 1
        rounds += 1
    for a, b in zip(plain, spec):
        assert a[:steps] == b[:steps]
    assert accepted > rounds and rounds < steps  # drafts were of use
