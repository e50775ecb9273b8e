"""Host side of the sequence operators (no GPU): what a call refuses before it
launches anything, workspace sizes, and the references' own checks."""
import ctypes as C

import numpy as np
import pytest

from tests import seqref

P = 1 << 20  # an aligned address that no refused call follows


@pytest.fixture(scope="module")
def stq():
    import linear_attention_recurrent_stq_amd as m
    return m


def _rule(stq, **kw):
    r = stq.StqRule(4, 128, 128, stq.GATE_SCALAR, stq.BF16)
    for n, x in kw.items():
        setattr(r, n, x)
    return r


RULES = [({"H": 0}, 1), ({"H": 4097}, 1), ({"d_k": 96}, 2), ({"d_v": 256}, 2), ({"gate": 2}, 1),
         ({"io_dtype": 2}, 1), ({"io_dtype": 0}, 1)]


def _step(stq, rule, **kw):
    x = dict(B=2, N=4, cu=P, q=P, k=P, v=P, a=P, beta=P, state=P, slots=3, ids=P, commit=P, o=P)
    x.update(kw)
    return stq.library().stq_recurrent_step(
        None if rule is None else C.byref(rule), x["B"], x["N"], x["cu"], x["q"], x["k"], x["v"], x["a"],
        x["beta"], x["state"], x["slots"], x["ids"], x["commit"], x["o"], None)


@pytest.mark.parametrize("bad,status", RULES)
def test_recurrent_refuses_a_rule(stq, bad, status):
    assert _step(stq, _rule(stq, **bad)) == status
    assert stq.library().stq_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    ({"B": -1}, 1), ({"N": -1}, 1), ({"slots": 1}, 1), ({"slots": -1}, 1), ({"cu": None}, 1), ({"q": None}, 1),
    ({"k": None}, 1), ({"v": None}, 1), ({"a": None}, 1), ({"beta": None}, 1), ({"state": None}, 1), ({"o": None}, 1),
    ({"q": P + 8}, 4), ({"o": P + 4}, 4), ({"state": P + 8}, 4), ({"cu": P + 2}, 4), ({"ids": P + 1}, 4),
    ({"commit": P + 2}, 4), ({"B": (1 << 18) + 1, "slots": 1 << 19}, 2)])
def test_recurrent_refuses_arguments(stq, kw, status):
    assert _step(stq, _rule(stq), **kw) == status
    assert stq.library().stq_last_error().decode()


def test_recurrent_nothing_to_do(stq):
    assert _step(stq, None) == 1
    assert _step(stq, _rule(stq), B=0, cu=None) == stq.STQ_OK
    assert _step(stq, _rule(stq), N=0, cu=None) == stq.STQ_OK


def _verify(stq, **kw):
    x = dict(B=2, T=3, V=100, dtype=1, tok=P, len=P, p=P, q=P, u=P, acc=P, nxt=P, ws=P, n=1 << 20)
    x.update(kw)
    return stq.library().stq_verify_draft(x["B"], x["T"], x["V"], x["dtype"], x["tok"], x["len"], x["p"], x["q"],
                                          x["u"], x["acc"], x["nxt"], x["ws"], x["n"], None)


@pytest.mark.parametrize("kw,status", [
    ({"B": -1}, 1), ({"T": -1}, 1), ({"V": 0}, 1), ({"dtype": 2}, 1), ({"B": 70000}, 2), ({"V": (1 << 30) + 1}, 2),
    ({"tok": None}, 1), ({"p": None}, 1), ({"q": None}, 1), ({"u": None}, 1), ({"acc": None}, 1), ({"nxt": None}, 1),
    ({"ws": None}, 1), ({"n": 31}, 3), ({"p": P + 4}, 4), ({"q": P + 4}, 4), ({"ws": P + 8}, 4), ({"tok": P + 2}, 4),
    ({"len": P + 2}, 4)])
def test_verify_refuses_arguments(stq, kw, status):
    assert _verify(stq, **kw) == status
    assert stq.library().stq_last_error().decode()


def test_verify_workspace(stq):
    n = C.c_size_t()
    for B, V, segs in ((1, 1, 1), (3, 2048, 1), (3, 2049, 2), (2, 129281, 64), (1, 1 << 20, 64)):
        assert stq.library().stq_verify_workspace(B, V, C.byref(n)) == 0
        assert 0 < n.value <= B * 64 * 16 and n.value >= B * (segs if V < 131072 else 1) * 16
    assert stq.library().stq_verify_workspace(1, 10, None) == 1
    assert _verify(stq, B=0) == stq.STQ_OK


def _forward(stq, rule, **kw):
    x = dict(B=2, N=200, cu=P, q=P, k=P, v=P, a=P, beta=P, first=P, o=P, last=P, ws=P, n=1 << 40)
    x.update(kw)
    return stq.library().stq_chunk_forward(
        None if rule is None else C.byref(rule), x["B"], x["N"], x["cu"], x["q"], x["k"], x["v"], x["a"], x["beta"],
        x["first"], x["o"], x["last"], x["ws"], x["n"], None)


def _backward(stq, rule, **kw):
    x = dict(B=2, N=200, cu=P, q=P, k=P, v=P, a=P, beta=P, first=P, do=P, dlast=P, dq=P, dk=P, dv=P, da=P, dbeta=P,
             dfirst=P, ws=P, n=1 << 40)
    x.update(kw)
    return stq.library().stq_chunk_backward(
        None if rule is None else C.byref(rule), x["B"], x["N"], x["cu"], x["q"], x["k"], x["v"], x["a"], x["beta"],
        x["first"], x["do"], x["dlast"], x["dq"], x["dk"], x["dv"], x["da"], x["dbeta"], x["dfirst"], x["ws"], x["n"],
        None)


def _workspace(stq, rule, B, N, backward):
    n = C.c_size_t()
    return stq.library().stq_chunk_workspace(C.byref(rule), B, N, backward, C.byref(n)), n.value


@pytest.mark.parametrize("bad,status", RULES)
def test_chunk_refuses_a_rule(stq, bad, status):
    for call in (_forward, _backward):
        assert call(stq, _rule(stq, **bad)) == status
        assert stq.library().stq_last_error().decode()
        assert call(stq, None) == 1
    assert _workspace(stq, _rule(stq, **bad), 1, 1, 0)[0] == status


@pytest.mark.parametrize("kw,status", [
    ({"B": -1}, 1), ({"N": -1}, 1), ({"cu": None}, 1), ({"q": None}, 1), ({"k": None}, 1), ({"v": None}, 1),
    ({"a": None}, 1), ({"beta": None}, 1), ({"ws": None}, 1), ({"ws": P + 8}, 4), ({"q": P + 8}, 4), ({"k": P + 4}, 4),
    ({"beta": P + 4}, 4), ({"cu": P + 2}, 4), ({"first": P + 8}, 4), ({"n": 1000}, 3), ({"B": 1 << 29}, 2),
    ({"B": (1 << 13) + 1}, 2),
    ({"N": 64 << 16}, 2), ({"N": (1 << 31) - 1}, 2)])
def test_chunk_refuses_arguments(stq, kw, status):
    many = _rule(stq, H=128)             # heads enough for the last four
    for call in (_forward, _backward):
        assert call(stq, many, **kw) == status
        assert stq.library().stq_last_error().decode()


@pytest.mark.parametrize("kw,status", [({"o": None}, 1), ({"o": P + 2}, 4), ({"last": P + 4}, 4)])
def test_chunk_forward_refuses_outputs(stq, kw, status):
    assert _forward(stq, _rule(stq), **kw) == status


@pytest.mark.parametrize("name", ["do", "dq", "dk", "dv", "da", "dbeta"])
def test_chunk_backward_refuses_outputs(stq, name):
    assert _backward(stq, _rule(stq), **{name: None}) == 1
    assert _backward(stq, _rule(stq), **{name: P + 8}) == 4
    for states in ("dlast", "dfirst"):
        assert _backward(stq, _rule(stq), **{states: P + 4}) == 4


def test_chunk_nothing_to_do(stq):
    assert _forward(stq, _rule(stq), B=0, cu=None, ws=None) == stq.STQ_OK
    assert _backward(stq, _rule(stq), B=0, cu=None, ws=None) == stq.STQ_OK


@pytest.mark.parametrize("gate", [0, 1])
@pytest.mark.parametrize("backward", [0, 1])
def test_chunk_workspace(stq, gate, backward):
    """Grows with both numbers, so a plan holds every smaller batch; the size that it names is the
    one that a call asks for."""
    rule = _rule(stq, gate=gate, H=3)
    last = 0
    for N in (0, 1, 64, 1000, 1024, 2047, 2048, 5000, 20000, 100000):
        for B in (1, 2, 7, 1000, 2000):
            s, n = _workspace(stq, rule, B, N, backward)
            assert s == 0
            assert n >= _workspace(stq, rule, max(1, B // 2), N, backward)[1]
            assert n >= _workspace(stq, rule, B, N // 2, backward)[1]
            assert n >= _workspace(stq, rule, B, max(0, N - 1), backward)[1]
        assert n >= last
        last = n
    call = _backward if backward else _forward
    assert call(stq, rule, n=_workspace(stq, rule, 2, 200, backward)[1] - 1) == 3
    assert stq.library().stq_chunk_workspace(C.byref(rule), 1, 1, backward, None) == 1
    assert _workspace(stq, rule, -1, 1, backward)[0] == 1 and _workspace(stq, rule, 1, -1, backward)[0] == 1


def test_reference_gradients_against_differences():
    rng = np.random.default_rng(0)
    for keyvec in (False, True):
        cu, H, dk, dv = [0, 3, 3, 8], 2, 3, 4
        x = {"q": rng.normal(size=(8, H, dk)), "k": rng.normal(size=(8, H, dk)) * 0.5,
             "v": rng.normal(size=(8, H, dv)), "beta": rng.uniform(0.1, 0.9, (8, H)),
             "a": rng.uniform(0.3, 1, (8, H, dk) if keyvec else (8, H)), "state": rng.normal(size=(3, H, dk, dv))}
        do, dl = rng.normal(size=(8, H, dv)), rng.normal(size=(3, H, dk, dv))

        def loss(y):
            o, last, _ = seqref.forward(cu, y["q"], y["k"], y["v"], y["a"], y["beta"], y["state"])
            return (o * do).sum() + (last * dl).sum()

        g = seqref.backward(cu, x["q"], x["k"], x["v"], x["a"], x["beta"], x["state"], do, dl)
        for n in x:
            for i in rng.choice(x[n].size, 12, replace=False):
                d = np.zeros(x[n].size)
                d[i] = 1e-6
                hi, lo = (loss(dict(x, **{n: x[n] + s * d.reshape(x[n].shape)})) for s in (1, -1))
                # central difference: truncation ~ 1e-12, cancellation ~ 1e-15 |loss| / 1e-6
                assert abs((hi - lo) / 2e-6 - g[n].ravel()[i]) < 1e-6 * max(1.0, abs(g[n].ravel()[i]))
