"""The status word of the score kernels: one a device, whatever the first call is part of."""
import subprocess
import sys
import textwrap

import pytest
import torch


def test_status_word_refuses_a_null_pointer():
    from ivf_quantizer_b200 import _lib
    assert _lib.LIB.fgmm_mx4_status_word(None) == _lib.ERR_INVALID_ARG


def _index(n, d, seed):
    import ivf_quantizer_b200 as q
    return q.MX4(torch.randn(n, d, generator=torch.Generator().manual_seed(seed)).cuda())


@pytest.fixture
def status_args(monkeypatch):
    """The status pointers that scores hand to the library, from a first call on."""
    from ivf_quantizer_b200 import mx4
    seen, call = [], mx4.call

    def record(fn, name, device, *args):
        if name == "fgmm_mx4_scores":
            seen.append(args[-1])
        call(fn, name, device, *args)

    monkeypatch.setattr(mx4, "call", record)
    monkeypatch.setattr(mx4, "_words", {})
    return seen


@pytest.mark.gpu
def test_first_scores_in_inference_mode(status_args):
    from ivf_quantizer_b200 import _lib, mx4
    index, queries = _index(300, 64, 1), _index(3, 64, 2)
    with torch.inference_mode():
        index.scores(queries)
    word = mx4._words[index.codes.device.index]
    assert status_args == [word.data_ptr()]
    word.fill_(_lib.ERR_TIMEOUT)
    with pytest.raises(_lib.FgmmError):
        index.check_status()
    assert index.status() == _lib.OK
    word.fill_(_lib.ERR_TIMEOUT)
    with torch.inference_mode():
        assert index.status() == _lib.ERR_TIMEOUT and index.status() == _lib.OK


@pytest.mark.gpu
def test_first_scores_in_a_captured_graph(status_args):
    from ivf_quantizer_b200 import _lib, mx4
    index, queries = _index(300, 64, 3), _index(3, 64, 4)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = index.scores(queries)
    word = mx4._words[index.codes.device.index]
    assert status_args == [word.data_ptr()]             # the kernel in the graph has it
    graph.replay()
    assert index.status() == _lib.OK
    assert torch.equal(out, index.scores(queries)) and status_args[1] == status_args[0]
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        with pytest.raises(RuntimeError):
            index.status()
        index.scores(queries)


@pytest.mark.gpu
def test_two_first_calls_have_one_word(status_args, monkeypatch):
    from ivf_quantizer_b200 import mx4

    class Late(dict):                                   # both callers look before either has stored
        def get(self, *_):
            return None

    monkeypatch.setattr(mx4, "_words", Late())
    index, queries = _index(300, 64, 5), _index(3, 64, 6)
    index.scores(queries)
    index.scores(queries)
    assert status_args[0] == status_args[1]


@pytest.mark.gpu
def test_everything_captured_in_a_fresh_process():
    """Codes made, scored and drawn from for the first time inside a capture."""
    code = """
        import torch
        import ivf_quantizer_b200 as q
        x = torch.randn(300, 64, device="cuda")
        qs, u = torch.randn(3, 64, device="cuda"), torch.full((3,), 0.5, device="cuda", dtype=torch.float64)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            index = q.MX4(x)
            s = index.scores(qs)
            ids, prob = q.sample_logits(s, u)
        x.copy_(x.flip(0))
        graph.replay()
        torch.cuda.synchronize()
        index.check_status()
        again = q.MX4(x)
        assert torch.equal(again.codes, index.codes) and torch.equal(again.scores(qs), s)
        a, b = q.sample_logits(s, u)
        assert torch.equal(a, ids) and torch.equal(b, prob)
    """
    r = subprocess.run([sys.executable, "-c", textwrap.dedent(code)], capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr


@pytest.mark.gpu
def test_a_report_reaches_every_index_of_the_device():
    from ivf_quantizer_b200 import _lib, mx4
    a, b, queries = _index(300, 64, 7), _index(200, 64, 8), _index(3, 64, 9)
    a.scores(queries), b.scores(queries)
    assert a.status() == b.status() == _lib.OK
    word = mx4._words[a.codes.device.index]
    word.fill_(_lib.ERR_TIMEOUT)
    c = _index(100, 64, 10)                             # made before anyone has read it
    assert a.status() == _lib.ERR_TIMEOUT
    d = _index(100, 64, 11)                             # and after
    assert a.status() == _lib.OK and d.status() == _lib.OK
    assert b.status() == _lib.ERR_TIMEOUT and c.status() == _lib.ERR_TIMEOUT
    assert b.status() == _lib.OK and c.status() == _lib.OK and int(word) == 0


@pytest.mark.gpu
def test_a_report_noted_while_the_word_is_cleared_is_not_lost(monkeypatch):
    """The word set again, as by another stream's kernel, after it was read and before it is 0."""
    from ivf_quantizer_b200 import _lib, mx4
    a, b, queries = _index(300, 64, 12), _index(200, 64, 13), _index(3, 64, 14)
    a.scores(queries), b.scores(queries)
    word = mx4._words[a.codes.device.index]

    class Racing:
        def data_ptr(self):
            return word.data_ptr()

        def __int__(self):
            code = int(word)
            word.fill_(_lib.ERR_TIMEOUT)                # b's kernel gives up here
            return code

        def zero_(self):
            word.zero_()

    word.fill_(_lib.ERR_TIMEOUT)
    with monkeypatch.context() as patch:
        patch.setitem(mx4._words, a.codes.device.index, Racing())
        assert a.status() == _lib.ERR_TIMEOUT
    assert b.status() == _lib.ERR_TIMEOUT and b.status() == _lib.OK and a.status() == _lib.OK
