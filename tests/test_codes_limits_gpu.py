"""Codes, scores and draws at the ends of their ranges and as programs with several threads, streams and
graph branches use them.  Values are small integers where sums have to be exact: results are compared
bit by bit."""
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


def _ints(n, d, seed):
    """Integers of -6 .. 6 that the codes hold (their blocks' largest magnitude is 4 or 6)."""
    g = torch.Generator().manual_seed(seed)
    grid = torch.tensor([-6.0, -4, -3, -2, -1, 0, 1, 2, 3, 4, 6])
    x = grid[torch.randint(0, 11, (n, d), generator=g)]
    x[:, ::32] = 4.0
    return x.cuda()


@pytest.mark.parametrize("m,n", [(1, 3), (20, 130), (130, 130)])
def test_the_longest_rows(m, n):
    import ivf_quantizer_b200 as q
    d = 1 << 20
    x, qs = _ints(n, d, 1), _ints(m, d, 2)
    x[:, 4096:-4096] = 0                    # partial sums stay below 2^24
    index = q.MX4(x)
    assert torch.equal(index.decode(), x)
    want = qs.double() @ x.double().T
    assert want.abs().max() < 2 ** 24 and torch.equal(index.scores(qs).double(), want)
    with pytest.raises(q.FgmmError):
        q.MX4(torch.zeros(1, d + 1, device="cuda"))


def test_the_most_rows():
    """As vectors and as queries: tile indices, byte offsets and coordinates near 2^31."""
    import ivf_quantizer_b200 as q
    from ivf_quantizer_b200 import _lib
    n = _lib.MX4_MAX_ROWS
    at = [0, 5, 127, (1 << 30) + 77, (1 << 31) - 5000, n - 129, n - 128, n - 2, n - 1]
    x = torch.zeros(n, 1, dtype=torch.bfloat16, device="cuda")
    x[at, 0] = torch.arange(1, 10, device="cuda").bfloat16()
    index = q.MX4(x)
    del x
    out = index.decode(torch.bfloat16)
    small = q.MX4(out[at].float())
    assert torch.equal(out[at, 0].float(), small.decode()[:, 0]) and int((out != 0).sum()) == 9
    held = out[at, 0].float()
    del out
    two = torch.tensor([[2.0]], device="cuda")
    s = index.scores(two, dtype=torch.bfloat16)
    assert torch.equal(s[0, at].float(), 2 * held) and int((s != 0).sum()) == 9
    del s
    s = q.MX4(two).scores(index, dtype=torch.bfloat16)
    assert s.shape == (n, 1)
    assert torch.equal(s[at, 0].float(), 2 * held) and int((s != 0).sum()) == 9
    del s, index
    torch.cuda.empty_cache()                # (43 GB of codes)


def test_many_short_rows_drawn():
    import ivf_quantizer_b200 as q
    rows = 3_000_001
    x = torch.full((rows, 2), -float("inf"), device="cuda")
    side = torch.randint(0, 2, (rows,), generator=torch.Generator().manual_seed(3)).cuda()
    x[torch.arange(rows, device="cuda"), side] = 1.5
    u = torch.rand(rows, dtype=torch.float64, device="cuda")
    for kw in ({}, {"top_k": 1}, {"top_p": 0.5}):
        ids, prob = q.sample_logits(x, u, **kw)
        assert torch.equal(ids, side.int()) and bool((prob == 1).all())


def test_the_same_codes_on_both_sides():
    import ivf_quantizer_b200 as q
    m = q.MX4(_ints(700, 300, 4))
    s, x = m.scores(m), m.decode().double()
    assert torch.equal(s.double(), x @ x.T)


def test_captured_branches_and_copies_between_the_kernels():
    """Kernels that may start early, behind nodes of other kinds and behind other streams."""
    import ivf_quantizer_b200 as q
    x, qs = _ints(3000, 300, 5), _ints(150, 300, 6)
    src, bias = torch.zeros_like(qs), torch.zeros(3000, device="cuda")
    index, other = q.MX4(x), torch.cuda.Stream()
    index.scores(qs)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        moved = src.clone()                             # a copy
        coded = q.MX4(moved)
        back = coded.decode()
        other.wait_stream(here)
        with torch.cuda.stream(other):
            norms = torch.mul(back, back).sum(1)
            a = index.scores(coded, bias=bias)          # behind an event
        bias2 = bias * 2
        b = index.scores(coded, bias=bias2)             # behind an elementwise kernel
        here.wait_stream(other)
        c = index.scores(back, bias=bias)               # encodes again
        moved.zero_()                                   # after everything that reads it
    for k in (1.0, 2.0):
        src.copy_(qs * k)
        bias.fill_(k)
        graph.replay()
        want = (qs.double() * k) @ x.double().T
        assert torch.equal(a.double(), want + k) and torch.equal(b.double(), want + 2 * k)
        assert torch.equal(c, a) and torch.equal(norms, (qs * k).square().sum(1))


def test_several_threads_at_once():
    import ivf_quantizer_b200 as q
    index = q.MX4(_ints(20001, 200, 7))
    work = [(_ints(m, 200, 8 + m), torch.rand(m, dtype=torch.float64, device="cuda")) for m in (1, 30, 90, 300)]

    def once(qs, u):
        s = index.scores(qs)
        ids, prob = q.sample_logits(s, u, temperature=40.0, top_k=50, top_p=0.9, min_p=0.01)
        return s, ids, prob, index.decode()

    want = [once(*w) for w in work]
    torch.cuda.synchronize()
    bad, start = [], threading.Barrier(len(work))

    def run(w, e):
        with torch.cuda.stream(torch.cuda.Stream()):
            start.wait()
            for _ in range(20):
                got = once(*w)
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, e)) or index.status():
                    bad.append(len(w[1]))

    threads = [threading.Thread(target=run, args=a) for a in zip(work, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad
