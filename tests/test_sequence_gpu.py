"""The sequence operators against plain 64-bit references, at the sizes, masks
and tables where they can go wrong."""
import numpy as np
import pytest
import torch  # before the library: both then use the HIP runtime that torch loads

from tests import seqref

pytestmark = pytest.mark.gpu

E32 = 2.0 ** -24   # half a step of fp32, relative


@pytest.fixture(scope="module")
def stq():
    import linear_attention_recurrent_stq_amd as m
    return m


def _inputs(rng, n, H, dk, dv, keyvec, bf16, lo=0.7):
    """Packed inputs as torch device tensors and as the numpy values they hold."""
    def dev(x, t):
        y = torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(t)
        return y.cuda(), y.double().numpy()
    io = torch.bfloat16 if bf16 else torch.float32
    unit = lambda x: x / np.linalg.norm(x, axis=-1, keepdims=True)
    x = {"q": dev(unit(rng.normal(size=(n, H, dk))), io), "k": dev(unit(rng.normal(size=(n, H, dk))), io),
         "v": dev(rng.normal(size=(n, H, dv)), io),
         "a": dev(rng.uniform(lo, 1, (n, H, dk) if keyvec else (n, H)), torch.float32),
         "beta": dev(rng.uniform(0, 1, (n, H)), torch.float32)}
    return {m: y[0] for m, y in x.items()}, {m: y[1] for m, y in x.items()}


def _dev(x, t):
    return torch.from_numpy(np.asarray(x)).to(t).cuda()


def _cu(lens):
    at = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return at, torch.from_numpy(at).cuda()


def _rel(got, want):
    """Distance over the reference's norm, over all elements."""
    n = np.linalg.norm(want)
    return np.linalg.norm(np.asarray(got, np.float64) - want) / n if n else np.abs(got).max()


def _within(got, want, tol):
    r = float(_rel(got, want))
    assert r < tol


# ---------------------------------------------------------------- recurrent
# A token's sums have d_k / 8 terms in a lane and three cross-lane adds, then
# four more roundings: an error of at most (d_k / 8 + 7) E32 of the state's and
# the token's norm enters per token.  With |k| <= 1, beta <= 1 and a <= 1 the
# update does not enlarge an error of the state, so after T tokens it is within
# T times that; outputs are the state times |q| = 1.  The norms of state and
# tokens are of one size here, hence the factor 4 against the norm of the result.
def _step_tol(dk, T):
    return 4 * T * (dk / 8 + 7) * E32


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("keyvec,bf16", [(False, False), (False, True), (True, False), (True, True)])
def test_recurrent(stq, dk, dv, keyvec, bf16):
    rng = np.random.default_rng(dk + dv)
    lens, H, slots = [1, 0, 5, 16, 2], 3, 7
    at, cu = _cu(lens)
    n = at[-1] + 3                       # three tokens behind the last sequence
    x, y = _inputs(rng, n, H, dk, dv, keyvec, bf16)
    ids = np.array([4, 0, 6, 1, 3], np.int32)
    S0 = rng.normal(size=(slots, H, dk, dv)).astype(np.float32)
    commit = np.array([1, 0, 2, 99, -1], np.int32)
    o = torch.full((n, H, dv), 7.0, device="cuda")
    for given in (None, commit):
        S = torch.from_numpy(S0).cuda()
        stq.recurrent_step(S, _dev(ids, torch.int32), cu, x["q"], x["k"], x["v"], x["a"], x["beta"], o,
                           commit=None if given is None else _dev(given, torch.int32))
        wo, last, kept = seqref.forward(at, *(y[m] for m in ("q", "k", "v", "a", "beta")), S0[ids],
                                        np.clip(commit, 0, lens))
        want = S0.astype(np.float64)
        want[ids] = last if given is None else kept
        go, gS = o.cpu().numpy(), S.cpu().numpy()
        assert (go[at[-1]:] == 7).all()
        _within(go[:at[-1]], wo[:at[-1]], _step_tol(dk, max(lens)))
        _within(gS, want, _step_tol(dk, max(lens)))
        for s in range(slots):           # untouched slots keep their bits
            if s not in ids or lens[list(ids).index(s)] == 0 or (given is not None and s == 3):
                assert np.array_equal(gS[s], S0[s]), s


def test_recurrent_equals_single_tokens_and_decode(stq):
    """Several tokens in one call, the same tokens one call each, and the
    decode step on fp32 units: the first two are the same bits, the third the
    same rule in another order of sums."""
    rng = np.random.default_rng(3)
    H, d, T, B = 4, 128, 4, 3
    at, cu = _cu([T] * B)
    x, y = _inputs(rng, T * B, H, d, d, True, True)
    S0 = torch.from_numpy(rng.normal(size=(B, H, d, d)).astype(np.float32)).cuda()
    S, o = S0.clone(), torch.empty(T * B, H, d, device="cuda")
    stq.recurrent_step(S, None, cu, x["q"], x["k"], x["v"], x["a"], x["beta"], o)
    L = stq.Layout(H, d, d, np.full(H, 32, np.uint8), gate=stq.GATE_KEYVEC)
    pool = stq.Pool(L, B)
    ids = torch.arange(B, dtype=torch.int32, device="cuda")
    stq.pack(pool, ids, S0)
    S1, one, od = S0.clone(), torch.empty(B, H, d, device="cuda"), torch.empty(B, H, d, device="cuda")
    cu1 = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    for t in range(T):
        z = {m: x[m].view(B, T, *x[m].shape[1:])[:, t].contiguous() for m in x}
        stq.recurrent_step(S1, ids, cu1, z["q"], z["k"], z["v"], z["a"], z["beta"], one)
        assert torch.equal(one, o.view(B, T, H, d)[:, t])
        stq.decode_step(pool, ids, z["q"], z["k"], z["v"], z["a"], z["beta"], od)
        _within(od.cpu().numpy(), one.double().cpu().numpy(), 2 * _step_tol(d, T))
    assert torch.equal(S, S1)


@pytest.mark.parametrize("keyvec", [False, True])
def test_recurrent_resets_and_bad_slots(stq, keyvec):
    """Gates of 0 drop the state exactly, beta 0 writes nothing, a slot id out
    of range gives NaN outputs and leaves every state."""
    rng = np.random.default_rng(5)
    H, d = 2, 64
    at, cu = _cu([3, 2, 1])
    x, y = _inputs(rng, 6, H, d, d, keyvec, False)
    x["a"][1] = 0
    x["beta"][2] = 0
    x["v"][5] = 0
    x["beta"][3:] = 0
    S0 = torch.from_numpy(rng.normal(size=(3, H, d, d)).astype(np.float32)).cuda()
    S, o = S0.clone(), torch.empty(6, H, d, device="cuda")
    stq.recurrent_step(S, _dev(np.array([2, 3, 0], np.int32), torch.int32), cu, x["q"], x["k"], x["v"], x["a"],
                       x["beta"], o)
    assert torch.isnan(o[3:5]).all() and torch.equal(S[1], S0[1])
    # after the reset the state is k u^T of that token alone, then decayed
    a2 = x["a"][2][:, :, None] if keyvec else x["a"][2][:, None, None]
    u = x["beta"][1][:, None] * x["v"][1]
    want = a2 * (x["k"][1][:, :, None] * u[:, None, :])
    assert torch.equal(S[2], want)
    a5 = x["a"][5][:, :, None] if keyvec else x["a"][5][:, None, None]
    assert torch.equal(S[0], a5 * S0[0])


def test_recurrent_python_refusals(stq):
    H, d = 2, 64
    x, _ = _inputs(np.random.default_rng(0), 2, H, d, d, False, False)
    S, o = torch.zeros(2, H, d, d, device="cuda"), torch.zeros(2, H, d, device="cuda")
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    good = dict(state=S, slot_ids=None, cu_seqlens=cu, o=o, **x)
    for bad in (dict(state=S[0]), dict(o=o.double()), dict(cu_seqlens=cu.long()), dict(cu_seqlens=cu.cpu()),
                dict(k=x["k"].bfloat16()), dict(q=x["q"].half()), dict(v=x["v"].transpose(1, 2)),
                dict(beta=x["beta"][:1]), dict(commit=cu), dict(slot_ids=cu), dict(state=S[:1]), dict(o=o.cpu())):
        with pytest.raises((ValueError, stq.StqError)):
            stq.recurrent_step(**{**good, **bad})
    stq.recurrent_step(**good)


# ------------------------------------------------------------------ chunks
# Errors of the chunked form, relative to the norm of the result.  A chunk's
# matrix products take operands of 22 bits, relative to the largest value of
# their row or column (which is up to sqrt(128) of its root mean square: 3.5
# bits), and sum 128 of them in fp32 in an order that the matrix units choose
# (at most 128 E32, in practice its root).  Six products stand one behind another,
# and the state passes through the chunks without enlarging an error (|k| <= 1,
# beta <= 1, a <= 1), a chunk's own errors adding to it.  So a result is within
# chunks * 6 * (2^-22 * 2^3.5 + 128 E32) of its norm; the outputs are then
# rounded to their type.
def _chunk_tol(lens):
    chunks = max(1, -(-max(lens) // 64))
    return chunks * 6 * (2.0 ** -18.5 + 128 * E32)


def _io_step(bf16):
    return 2.0 ** -8 if bf16 else E32


LENS = {"one": [1], "short": [3, 0, 17, 64, 1], "edge": [63, 65, 128, 127, 129, 0], "long": [500, 31]}


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("keyvec,bf16", [(False, False), (False, True), (True, False), (True, True)])
def test_chunk_forward(stq, lens, dk, dv, keyvec, bf16):
    rng = np.random.default_rng(dk + 2 * dv)
    lens, H = LENS[lens], 2
    at, cu = _cu(lens)
    n, B = at[-1] + 2, len(lens)         # two tokens behind the last sequence
    x, y = _inputs(rng, n, H, dk, dv, keyvec, bf16)
    S0 = rng.normal(size=(B, H, dk, dv)).astype(np.float32)
    S = torch.from_numpy(S0).cuda()
    plan = stq.ChunkPlan(H, dk, dv, gate=int(keyvec), io_dtype=stq.BF16 if bf16 else stq.F32, max_tokens=n + 70,
                         max_seqs=B + 1)
    plan.workspace.fill_(255)            # what the workspace held does not matter
    o = torch.full_like(x["v"], 7.0)
    last = torch.full_like(S, 7.0)
    ins = (cu, x["q"], x["k"], x["v"], x["a"], x["beta"])
    stq.chunk_forward(plan, *ins, o, initial_state=S, final_state=last)
    wo, wl, _ = seqref.forward(at, *(y[m] for m in ("q", "k", "v", "a", "beta")), S0)
    go = o.double().cpu().numpy()
    assert (go[at[-1]:] == 7).all()
    _within(go[:at[-1]], wo[:at[-1]], _chunk_tol(lens) + _io_step(bf16))
    _within(last.cpu().numpy(), wl, _chunk_tol(lens))
    for b in range(B):                   # sequence by sequence: a small one is not lost in a large one
        _within(last[b].cpu().numpy(), wl[b], _chunk_tol(lens))
        if lens[b] == 0:
            assert torch.equal(last[b], S[b])
    # in place, the same bits; without states, from zero
    o2 = torch.zeros_like(o)
    stq.chunk_forward(plan, *ins, o2, initial_state=S, final_state=S)
    assert torch.equal(o2[:at[-1]], o[:at[-1]]) and torch.equal(S, last)
    stq.chunk_forward(plan, *ins, o2)
    wo, _, _ = seqref.forward(at, *(y[m] for m in ("q", "k", "v", "a", "beta")), np.zeros_like(S0))
    _within(o2.double().cpu().numpy()[:at[-1]], wo[:at[-1]], _chunk_tol(lens) + _io_step(bf16))


@pytest.mark.parametrize("keyvec,bf16", [(False, False), (False, True), (True, False), (True, True)])
@pytest.mark.parametrize("what", ["resets", "strong", "beta0", "tiny", "large", "same keys", "zero"])
def test_chunk_forward_extremes(stq, keyvec, bf16, what):
    """Gates of 0 and gates that underflow over a chunk, write strengths of 0
    and 1, values and states of extreme size, keys that are all the same, and
    all zeros."""
    rng = np.random.default_rng(11)
    lens, H, d = [150, 64], 3, 128
    at, cu = _cu(lens)
    n = at[-1]
    x, y = _inputs(rng, n, H, d, d, keyvec, bf16)
    S0 = rng.normal(size=(2, H, d, d)).astype(np.float32)
    if what == "resets":
        x["a"][::7] = 0.0
    elif what == "strong":
        x["a"].mul_(1e-3)
        x["a"][:, 1] = 1.0
        x["a"][5:9] = 1e-30
    elif what == "beta0":
        x["beta"][::2] = 0.0
        x["beta"][1::4] = 1.0
        x["beta"][3] = 1e-20
    elif what == "tiny":
        for m in ("v", "q"):
            x[m].mul_(2.0 ** -60)
        x["k"][::3].mul_(2.0 ** -40)
        S0 *= np.float32(2.0 ** -60)
    elif what == "large":
        x["v"].mul_(2.0 ** 60)
        x["q"].mul_(2.0 ** 30)
        x["v"][:, :, 3].mul_(2.0 ** -50)
        S0 *= np.float32(2.0 ** 60)
    elif what == "same keys":
        x["k"][:] = x["k"][0]
    else:
        for m in ("q", "k", "v", "beta"):
            x[m].zero_()
        S0[:] = 0
    y = {m: t.double().cpu().numpy() for m, t in x.items()}
    S = torch.from_numpy(S0).cuda()
    plan = stq.ChunkPlan(H, d, d, gate=int(keyvec), io_dtype=stq.BF16 if bf16 else stq.F32, max_tokens=n, max_seqs=2)
    o, last = torch.empty_like(x["v"]), torch.empty_like(S)
    stq.chunk_forward(plan, cu, x["q"], x["k"], x["v"], x["a"], x["beta"], o, initial_state=S, final_state=last)
    wo, wl, _ = seqref.forward(at, *(y[m] for m in ("q", "k", "v", "a", "beta")), S0)
    _within(o.double().cpu().numpy(), wo, _chunk_tol(lens) + _io_step(bf16))
    _within(last.cpu().numpy(), wl, _chunk_tol(lens))
    if what == "large":                  # a small column keeps its own accuracy
        _within(o.double().cpu().numpy()[:, :, 3], wo[:, :, 3], _chunk_tol(lens) + _io_step(bf16))


def test_chunk_forward_sequences_apart(stq):
    """A NaN or infinity in one sequence and head stays there; a sequence gives the
    same bits alone and in a batch; a bad table of starts writes nothing outside."""
    rng = np.random.default_rng(2)
    lens, H, d = [100, 70, 1], 2, 128
    at, cu = _cu(lens)
    x, _ = _inputs(rng, at[-1], H, d, d, True, True)
    ins = [x[m] for m in ("q", "k", "v", "a", "beta")]
    plan = stq.ChunkPlan(H, d, d, gate=1, max_tokens=at[-1], max_seqs=3)
    o, last = torch.empty_like(x["v"]), torch.empty(3, H, d, d, device="cuda")
    stq.chunk_forward(plan, cu, *ins, o, final_state=last)
    x["v"][at[1] + 3, 0, 5] = float("nan")
    x["k"][at[1] + 9, 0, 5] = float("inf")
    o2, last2 = torch.empty_like(o), torch.empty_like(last)
    stq.chunk_forward(plan, cu, *ins, o2, final_state=last2)
    assert torch.isnan(last2[1, 0]).any()
    for t, t2 in ((o, o2), (last, last2)):
        lo, hi = (at[1], at[2]) if t is o else (1, 2)
        assert torch.equal(t[:lo], t2[:lo]) and torch.equal(t[hi:], t2[hi:]) and torch.equal(t[lo:hi, 1], t2[lo:hi, 1])
    one = torch.empty_like(o)[:lens[0]]
    l1 = torch.empty(1, H, d, d, device="cuda")
    stq.chunk_forward(plan, cu[:2], *[t[:lens[0]] for t in ins], one, final_state=l1)
    assert torch.equal(one, o[:lens[0]]) and torch.equal(l1[0], last[0])
    guard = torch.full((at[-1] + 64, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    for bad in ([-5, 400, 20, 90], [171, 0, 171, 0], [3, 2, 1, 0]):
        stq.chunk_forward(plan, _dev(np.array(bad, np.int32), torch.int32), *ins, guard[:at[-1]], final_state=last2)
        assert (guard[at[-1]:] == 7).all()


# A long sequence, alone or with few others, passes in segments: a segment's end from no state
# and its matrix are each within the tolerance of a state passing through it, hence twice that.
@pytest.mark.parametrize("lens", [[3500], [4000, 2300], [9300, 5, 0]])
@pytest.mark.parametrize("dk,dv,keyvec,bf16", [(64, 128, False, False), (128, 64, False, True), (64, 64, True, False),
                                               (128, 128, True, True), (128, 128, False, True)])
def test_chunk_forward_long(stq, lens, dk, dv, keyvec, bf16):
    rng = np.random.default_rng(dk + 5 * dv)
    H = 1
    at, cu = _cu(lens)
    n, B = at[-1] + 2, len(lens)
    x, y = _inputs(rng, n, H, dk, dv, keyvec, bf16, lo=0.998)
    S0 = rng.normal(size=(B, H, dk, dv)).astype(np.float32)
    S = torch.from_numpy(S0).cuda()
    plan = stq.ChunkPlan(H, dk, dv, gate=int(keyvec), io_dtype=stq.BF16 if bf16 else stq.F32, max_tokens=n + 70,
                         max_seqs=B + 1)
    plan.workspace.fill_(255)
    o, last = torch.full_like(x["v"], 7.0), torch.full_like(S, 7.0)
    ins = (cu, x["q"], x["k"], x["v"], x["a"], x["beta"])
    stq.chunk_forward(plan, *ins, o, initial_state=S, final_state=last)
    wo, wl, _ = seqref.forward(at, *(y[m] for m in ("q", "k", "v", "a", "beta")), S0)
    go = o.double().cpu().numpy()
    assert (go[at[-1]:] == 7).all()
    _within(go[:at[-1]], wo[:at[-1]], 2 * _chunk_tol(lens) + _io_step(bf16))
    for t in range(0, at[-1], 500):      # no part is lost in the whole
        e = min(t + 500, at[-1])
        _within(go[t:e], wo[t:e], 2 * _chunk_tol(lens) + _io_step(bf16))
    for b in range(B):
        _within(last[b].cpu().numpy(), wl[b], 2 * _chunk_tol(lens))
        if lens[b] == 0:
            assert torch.equal(last[b], S[b])
    # in place and again, the same bits; without states, from zero
    o2 = torch.zeros_like(o)
    stq.chunk_forward(plan, *ins, o2, initial_state=S, final_state=S)
    assert torch.equal(o2[:at[-1]], o[:at[-1]]) and torch.equal(S, last)
    stq.chunk_forward(plan, *ins, o2)
    wo, _, _ = seqref.forward(at, *(y[m] for m in ("q", "k", "v", "a", "beta")), np.zeros_like(S0))
    _within(o2.double().cpu().numpy()[:at[-1]], wo[:at[-1]], 2 * _chunk_tol(lens) + _io_step(bf16))


def test_chunk_forward_then_steps(stq):
    """The pieces together: a prompt by chunks, its last tokens one by one from
    the state it left, against the whole sequence at once."""
    rng = np.random.default_rng(8)
    H, d, B, n = 4, 128, 3, 140
    at, cu = _cu([n] * B)
    x, y = _inputs(rng, B * n, H, d, d, False, True)
    v = {m: x[m].view(B, n, *x[m].shape[1:]) for m in x}
    plan = stq.ChunkPlan(H, d, d, max_tokens=B * n, max_seqs=B)
    cut = 133
    head = [v[m][:, :cut].reshape(B * cut, *x[m].shape[1:]).contiguous() for m in ("q", "k", "v", "a", "beta")]
    tail = [v[m][:, cut:].reshape(B * (n - cut), *x[m].shape[1:]).contiguous() for m in ("q", "k", "v", "a", "beta")]
    S = torch.empty(B, H, d, d, device="cuda")
    o1 = torch.empty_like(head[2])
    stq.chunk_forward(plan, _cu([cut] * B)[1], *head, o1, final_state=S)
    o2 = torch.empty(B * (n - cut), H, d, device="cuda")
    stq.recurrent_step(S, None, _cu([n - cut] * B)[1], *tail, o2)
    wo, wl, _ = seqref.forward(at, *(y[m] for m in ("q", "k", "v", "a", "beta")), np.zeros((B, H, d, d)))
    wo = wo.reshape(B, n, H, d)
    tol = _chunk_tol([n]) + _step_tol(d, n - cut)
    _within(o2.cpu().numpy().reshape(B, n - cut, H, d), wo[:, cut:], tol)
    _within(S.cpu().numpy(), wl, tol)
    _within(o1.double().cpu().numpy().reshape(B, cut, H, d), wo[:, :cut], tol + 2.0 ** -8)


@pytest.mark.parametrize("kw", [{}, {"window": 4}, {"scale_fit": 1}])
def test_serving(stq, kw):
    """A request's whole life: its prompt in two parts into a pool of fp32 and 8-bit units, decode
    steps from there; drafted tokens run ahead on the fp32 states, checked, and committed."""
    rng = np.random.default_rng(21)
    H, d, B, slots = 4, 128, 3, 5
    lens, tail = [130, 1, 77], 4
    at, cu = _cu(lens)
    n = at[-1]
    x, y = _inputs(rng, n, H, d, d, True, True)
    names = ("q", "k", "v", "a", "beta")
    bits = np.full(H, 8, np.uint8) if kw else np.array([32, 32, 8, 32], np.uint8)
    L = stq.Layout(H, d, d, bits, gate=stq.GATE_KEYVEC, **kw)
    pool, plan = stq.Pool(L, slots), stq.ChunkPlan(H, d, d, gate=1, max_tokens=n, max_seqs=B)
    ids = torch.tensor([4, 0, 2], dtype=torch.int32, device="cuda")
    states, o = torch.empty(B, H, d, d, device="cuda"), torch.empty_like(x["v"])
    stq.prefill(pool, plan, ids, cu, *[x[m] for m in names], o, states)
    wo, wl, _ = seqref.forward(at, *(y[m] for m in names), np.zeros((B, H, d, d)))
    _within(o.double().cpu().numpy(), wo, _chunk_tol(lens) + 2.0 ** -8)
    _within(states.cpu().numpy(), wl, _chunk_tol(lens))
    # the pool holds what packing these states gives, and the next part begins from it
    held, other = torch.empty_like(states), stq.Pool(L, slots)
    stq.unpack(pool, ids, held)
    stq.pack(other, ids, states)
    again = torch.empty_like(states)
    stq.unpack(other, ids, again)
    assert torch.equal(held, again)
    x2, y2 = _inputs(rng, n, H, d, d, True, True)
    stq.prefill(pool, plan, ids, cu, *[x2[m] for m in names], o, states, resume=True)
    wo, wl, _ = seqref.forward(at, *(y2[m] for m in names), held.double().cpu().numpy())
    _within(o.double().cpu().numpy(), wo, _chunk_tol(lens) + 2.0 ** -8)
    _within(states.cpu().numpy(), wl, _chunk_tol(lens))
    # decode steps on the pool: the same as on the unpacked state while the units are fp32
    stq.unpack(pool, ids, held)
    x3, y3 = _inputs(rng, B, H, d, d, True, True)
    od = torch.empty(B, H, d, device="cuda")
    stq.decode_step(pool, ids, *[x3[m] for m in names], od)
    wo, _, _ = seqref.forward(list(range(B + 1)), *(y3[m] for m in names), held.double().cpu().numpy())
    if not kw:
        _within(od.cpu().numpy()[:, [0, 1, 3]], wo[:, [0, 1, 3]], _step_tol(d, 1))
    # drafted tokens: ahead of the states, accepted or not, then taken in
    T, V = tail, 37
    xd, yd = _inputs(rng, B * T, H, d, d, True, True)
    cud, S = _cu([T] * B)[1], states.clone()
    od = torch.empty(B * T, H, d, device="cuda")
    p = rng.random((B, T + 1, V)).astype(np.float32)
    q = rng.random((B, T, V)).astype(np.float32)
    p, q = p / p.sum(-1, keepdims=True), q / q.sum(-1, keepdims=True)
    tok, r = rng.integers(0, V, (B, T)).astype(np.int32), rng.random((B, T + 1)).astype(np.float32)
    acc, nxt = (torch.empty(B, dtype=torch.int32, device="cuda") for _ in range(2))
    check = stq.VerifyPlan(B, T, V)
    stq.recurrent_step(S, None, cud, *[xd[m] for m in names], od, commit=torch.zeros_like(acc))
    assert torch.equal(S, states)
    stq.verify_draft(check, _dev(tok, torch.int32), *[_dev(z, torch.float32) for z in (p, q, r)], acc, nxt)
    wa, _ = seqref.verify(tok, None, p, q, r)
    assert (acc.cpu().numpy() == wa).all()
    stq.recurrent_step(S, None, cud, *[xd[m] for m in names], od, commit=acc)
    _, _, kept = seqref.forward(np.arange(B + 1) * T, *(yd[m] for m in names), states.double().cpu().numpy(), wa)
    _within(S.cpu().numpy(), kept, _step_tol(d, T))


def test_prefill_refusals(stq):
    H, d, n = 2, 64, 5
    x, _ = _inputs(np.random.default_rng(0), n, H, d, d, False, True)
    cu = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    ids = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    pool = stq.Pool(stq.Layout(H, d, d, np.full(H, 8, np.uint8)), 2)
    plan = stq.ChunkPlan(H, d, d, max_tokens=n, max_seqs=2)
    S = torch.zeros(2, H, d, d, device="cuda")
    good = dict(pool=pool, plan=plan, slot_ids=ids, cu_seqlens=cu, o=torch.empty_like(x["v"]), states=S, **x)
    for bad in (dict(slot_ids=ids[:1]), dict(states=S[:1]), dict(states=None), dict(states=S.double()),
                dict(slot_ids=ids.long()), dict(plan=stq.ChunkPlan(H, d, d, gate=1, max_tokens=n, max_seqs=2)),
                dict(pool=stq.Pool(stq.Layout(H, d, 128, np.full(H, 8, np.uint8)), 2)), dict(o=good["o"][:2])):
        with pytest.raises((ValueError, stq.StqError)):
            stq.prefill(**{**good, **bad})
    stq.prefill(**good)


def test_chunk_forward_in_a_graph(stq):
    """Captured once, replayed on new inputs in place, with eager work between."""
    rng = np.random.default_rng(4)
    lens, H, d = [90, 64, 5], 2, 64
    at, cu = _cu(lens)
    plan = stq.ChunkPlan(H, d, d, gate=1, max_tokens=at[-1], max_seqs=3)
    other = stq.ChunkPlan(H, d, d, gate=1, max_tokens=at[-1], max_seqs=3)
    x, _ = _inputs(rng, at[-1], H, d, d, True, True)
    names = ("q", "k", "v", "a", "beta")
    o, S = torch.empty_like(x["v"]), torch.zeros(3, H, d, d, device="cuda")
    o2, S2 = torch.empty_like(o), torch.empty_like(S)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        stq.chunk_forward(plan, cu, *[x[m] for m in names], o, initial_state=S, final_state=S)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stq.chunk_forward(plan, cu, *[x[m] for m in names], o, initial_state=S, final_state=S)
    for i in range(4):
        new, _ = _inputs(rng, at[-1], H, d, d, True, True)
        for m in names:
            x[m].copy_(new[m])
        S2.copy_(S)
        stq.chunk_forward(other, cu, *[new[m] for m in names], o2, initial_state=S2, final_state=S2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(S, S2)


def test_chunk_forward_long_in_a_graph(stq):
    """The segments of a long sequence, captured once and replayed on other starts and values."""
    rng = np.random.default_rng(6)
    n, H, d = 3500, 2, 64
    plan, other = (stq.ChunkPlan(H, d, d, max_tokens=n, max_seqs=2) for _ in range(2))
    cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    x, _ = _inputs(rng, n, H, d, d, False, True, lo=0.99)
    names = ("q", "k", "v", "a", "beta")
    o, S = torch.zeros_like(x["v"]), torch.zeros(1, H, d, d, device="cuda")
    o2, S2 = torch.zeros_like(o), torch.empty_like(S)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        stq.chunk_forward(plan, cu, *[x[m] for m in names], o, initial_state=S, final_state=S)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        stq.chunk_forward(plan, cu, *[x[m] for m in names], o, initial_state=S, final_state=S)
    for i, length in enumerate((n, 3000, 5, 0)):
        new, _ = _inputs(rng, n, H, d, d, False, True, lo=0.99)
        for m in names:
            x[m].copy_(new[m])
        cu[1] = length
        S2.copy_(S)
        o.fill_(i)
        o2.fill_(i)
        stq.chunk_forward(other, cu, *[new[m] for m in names], o2, initial_state=S2, final_state=S2)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(S, S2)


def test_chunk_python_refusals(stq):
    H, d, n = 2, 64, 5
    x, _ = _inputs(np.random.default_rng(0), n, H, d, d, False, True)
    cu = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    plan = stq.ChunkPlan(H, d, d, max_tokens=n, max_seqs=2)
    S = torch.zeros(2, H, d, d, device="cuda")
    good = dict(plan=plan, cu_seqlens=cu, o=torch.empty_like(x["v"]), initial_state=S, final_state=S, **x)
    more = torch.zeros(4, dtype=torch.int32, device="cuda")
    for bad in (dict(cu_seqlens=more), dict(cu_seqlens=cu.long()), dict(o=good["o"].float()), dict(o=good["o"][:3]),
                dict(initial_state=S[:1]), dict(final_state=S.double()), dict(a=x["a"][:, :, None].expand(n, H, d)),
                dict(q=x["q"].float(), k=x["k"].float(), v=x["v"].float()), dict(k=x["k"][:, :1]),
                dict(plan=stq.ChunkPlan(H, d, d, max_tokens=4, max_seqs=2)),
                dict(plan=stq.ChunkPlan(H, d, 128, max_tokens=n, max_seqs=2))):
        with pytest.raises((ValueError, stq.StqError)):
            stq.chunk_forward(**{**good, **bad})
    stq.chunk_forward(**good)


# ----------------------------------------------------------------- backward
# Each gradient is one more product, and one more pass through the chunks, away from the
# inputs than an output: twice the products of the forward tolerance.  The
# gradient of a gate is a difference of sums over a chunk's 64 tokens divided by it
# (gates of 0.7 and more here): a factor sqrt(64) / 0.7, taken as 12.
def _grad_tol(name, lens):
    return 2 * _chunk_tol(lens) * (12 if name == "a" else 1)


def _grads(stq, at, cu, x, keyvec, bf16, S0, do, dlast, plan=None, **kw):
    H, dk, dv = x["q"].shape[1], x["q"].shape[2], x["v"].shape[2]
    B = len(at) - 1
    if plan is None:
        plan = stq.ChunkPlan(H, dk, dv, gate=int(keyvec), io_dtype=stq.BF16 if bf16 else stq.F32,
                             max_tokens=x["q"].shape[0], max_seqs=B, backward=True)
        plan.workspace.fill_(255)
    g = {m: torch.full_like(x[m], 7.0) for m in ("q", "k", "v", "a", "beta")}
    g["state"] = torch.full((B, H, dk, dv), 7.0, device="cuda")
    stq.chunk_backward(plan, cu, *[x[m] for m in ("q", "k", "v", "a", "beta")], do, g["q"], g["k"], g["v"], g["a"],
                       g["beta"], initial_state=S0, d_final_state=dlast, d_initial_state=g["state"], **kw)
    return g


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("keyvec,bf16", [(False, False), (False, True), (True, False), (True, True)])
def test_chunk_backward(stq, lens, dk, dv, keyvec, bf16):
    rng = np.random.default_rng(dk + 3 * dv)
    lens, H = LENS[lens], 2
    at, cu = _cu(lens)
    n, B = at[-1] + 2, len(lens)
    x, y = _inputs(rng, n, H, dk, dv, keyvec, bf16)
    io = torch.bfloat16 if bf16 else torch.float32
    do = torch.from_numpy(rng.normal(size=(n, H, dv)).astype(np.float32)).to(io)
    S0, dlast = (rng.normal(size=(B, H, dk, dv)).astype(np.float32) for _ in range(2))
    names = ("q", "k", "v", "a", "beta")
    for first, last in ((S0, dlast), (None, None)):
        g = _grads(stq, at, cu, x, keyvec, bf16, None if first is None else torch.from_numpy(first).cuda(), do.cuda(),
                   None if last is None else torch.from_numpy(last).cuda())
        zero = np.zeros_like(S0)
        want = seqref.backward(at, *(y[m] for m in names), zero if first is None else first, do.double().numpy(),
                               zero if last is None else last)
        for m in names:
            got = g[m].double().cpu().numpy()
            assert (got[at[-1]:] == 7).all()
            _within(got[:at[-1]], want[m][:at[-1]], _grad_tol(m, lens) + _io_step(bf16 and m in "qkv"))
        _within(g["state"].cpu().numpy(), want["state"], _grad_tol("state", lens))


# What the pairs must keep, as a root mean square: over many elements errors are independent.  A
# value's error as hi + lo is at most 2^-22 of it, evenly spread: 2^-22.8; two operands, the
# product of the lo parts that is left out (2^-23.6) and a sum of 128 terms in fp32 (2^-22.5):
# 2^-21.4 a product.  Six stand one behind another in a state or output, twelve in a gradient.
@pytest.mark.parametrize("keyvec,bf16", [(False, False), (False, True), (True, False), (True, True)])
def test_chunk_keeps_22_bits(stq, keyvec, bf16):
    rng = np.random.default_rng(17)
    n, H, d = 256, 2, 128
    at, cu = _cu([n])
    x, y = _inputs(rng, n, H, d, d, keyvec, bf16)
    names = ("q", "k", "v", "a", "beta")
    zero = np.zeros((1, H, d, d))
    plan = stq.ChunkPlan(H, d, d, gate=int(keyvec), io_dtype=stq.BF16 if bf16 else stq.F32, max_tokens=n, max_seqs=1,
                         backward=True)
    o, last = torch.empty_like(x["v"]), torch.empty(1, H, d, d, device="cuda")
    stq.chunk_forward(plan, cu, *[x[m] for m in names], o, final_state=last)
    wo, wl, _ = seqref.forward(at, *(y[m] for m in names), zero)
    _within(last.cpu().numpy(), wl, 6 ** 0.5 * 2.0 ** -21.4)
    do = torch.from_numpy(rng.normal(size=(n, H, d)).astype(np.float32)).to(x["v"].dtype)
    g = _grads(stq, at, cu, x, keyvec, bf16, None, do.cuda(), None, plan=plan)
    want = seqref.backward(at, *(y[m] for m in names), zero, do.double().numpy(), zero)
    for m in ("beta", "state"):
        _within(g[m].double().cpu().numpy(), want[m], 12 ** 0.5 * 2.0 ** -21.4)
    if not bf16:
        _within(o.double().cpu().numpy(), wo, 6 ** 0.5 * 2.0 ** -21.4)
        for m in ("q", "k", "v"):
            _within(g[m].double().cpu().numpy(), want[m], 12 ** 0.5 * 2.0 ** -21.4)


@pytest.mark.parametrize("keyvec", [False, True])
@pytest.mark.parametrize("what", ["strong", "beta0", "tiny", "same keys", "zero"])
def test_chunk_backward_extremes(stq, keyvec, what):
    rng = np.random.default_rng(21)
    lens, H, d = [150, 64], 2, 128
    at, cu = _cu(lens)
    x, _ = _inputs(rng, at[-1], H, d, d, keyvec, False)
    S0, dlast = (rng.normal(size=(2, H, d, d)).astype(np.float32) for _ in range(2))
    do = rng.normal(size=(at[-1], H, d)).astype(np.float32)
    if what == "strong":
        x["a"].mul_(0.05)
        x["a"][::3].mul_(0.05)
    elif what == "beta0":
        x["beta"][::2] = 0.0
        x["beta"][1::4] = 1.0
    elif what == "tiny":
        for m in ("v", "q"):
            x[m].mul_(2.0 ** -30)
        S0 *= np.float32(2.0 ** -30)
        do *= np.float32(2.0 ** -30)
        dlast *= np.float32(2.0 ** -60)
    elif what == "same keys":
        x["k"][:] = x["k"][0]
    elif what == "zero":
        for m in ("q", "k", "v", "beta"):
            x[m].zero_()
    y = {m: t.double().cpu().numpy() for m, t in x.items()}
    g = _grads(stq, at, cu, x, keyvec, False, torch.from_numpy(S0).cuda(), torch.from_numpy(do).cuda(),
               torch.from_numpy(dlast).cuda())
    want = seqref.backward(at, *(y[m] for m in ("q", "k", "v", "a", "beta")), S0, do, dlast)
    for m in g:
        got, w = g[m].cpu().numpy().astype(np.float64), want[m]
        if m == "a":                     # what is formed in sums is a times it
            got, w = got * y["a"], w * y["a"]
        _within(got, w, _grad_tol(m, lens))


@pytest.mark.parametrize("keyvec", [False, True])
def test_chunk_backward_against_differences(stq, keyvec):
    """Directional differences of the forward kernel's own loss: in fp32, so the
    outputs' errors (relative _chunk_tol of a loss of size sqrt(outputs)) over twice
    the step bound the comparison, beside the step's square."""
    rng = np.random.default_rng(31)
    lens, H, d = [70, 9], 2, 64
    at, cu = _cu(lens)
    x, _ = _inputs(rng, at[-1], H, d, d, keyvec, False)
    S0, dlast = (torch.from_numpy(rng.normal(size=(2, H, d, d)).astype(np.float32)).cuda() for _ in range(2))
    do = torch.from_numpy(rng.normal(size=(at[-1], H, d)).astype(np.float32)).cuda()
    names = ("q", "k", "v", "a", "beta")
    g = _grads(stq, at, cu, x, keyvec, False, S0, do, dlast)
    plan = stq.ChunkPlan(H, d, d, gate=int(keyvec), io_dtype=stq.F32, max_tokens=at[-1], max_seqs=2)

    def loss(z, S):
        o, last = torch.empty_like(x["v"]), torch.empty_like(S)
        stq.chunk_forward(plan, cu, *[z[m] for m in names], o, initial_state=S, final_state=last)
        return float((o.double() * do).sum() + (last.double() * dlast).sum()), float(
            (o.double() * do).norm() + (last.double() * dlast).norm())

    eps = 1e-2
    for m in names + ("state",):
        base = S0 if m == "state" else x[m]
        v = torch.from_numpy(rng.normal(size=tuple(base.shape)).astype(np.float32)).cuda()
        v *= 0.2 / v.abs().max()
        put = lambda s: (x, base + s * v) if m == "state" else (dict(x, **{m: base + s * v}), S0)
        (hi, size), (lo, _) = loss(*put(eps)), loss(*put(-eps))
        (hi2, _), (lo2, _) = loss(*put(eps / 2)), loss(*put(-eps / 2))
        d1, d2 = (hi - lo) / (2 * eps), (hi2 - lo2) / eps
        want = float((g[m].double() * v).sum())
        # d2's own truncation is a third of its distance from d1
        assert abs(d2 - want) < abs(d1 - d2) + 2 * _chunk_tol(lens) * size / eps


@pytest.mark.parametrize("lens,H,dk,dv,keyvec,bf16", [
    ([70, 3, 200], 16, 128, 128, True, True), ([70, 3, 200], 8, 128, 64, False, True),
    ([1, 0, 3, 2] * 300, 1, 64, 64, True, False), ([2, 1, 0] * 400, 2, 64, 128, False, True),
    ([1300], 1, 128, 128, False, False)])
def test_chunk_many_heads_and_sequences(stq, lens, H, dk, dv, keyvec, bf16):
    """Heads in groups of eight, more sequences than are put in order, a longer one; on another
    stream than the current one."""
    rng = np.random.default_rng(31)
    at, cu = _cu(lens)
    n, B = at[-1], len(lens)
    x, y = _inputs(rng, n, H, dk, dv, keyvec, bf16)
    S0, dlast = (rng.normal(size=(B, H, dk, dv)).astype(np.float32) for _ in range(2))
    do = torch.from_numpy(rng.normal(size=(n, H, dv)).astype(np.float32)).to(x["v"].dtype)
    names = ("q", "k", "v", "a", "beta")
    first, grad, dout = torch.from_numpy(S0).cuda(), torch.from_numpy(dlast).cuda(), do.cuda()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan = stq.ChunkPlan(H, dk, dv, gate=int(keyvec), io_dtype=stq.BF16 if bf16 else stq.F32, max_tokens=n, max_seqs=B,
                         backward=True)
    o, last = torch.full_like(x["v"], 7.0), torch.full_like(first, 7.0)
    torch.cuda.synchronize()
    stq.chunk_forward(plan, cu, *[x[m] for m in names], o, initial_state=first, final_state=last, stream=side)
    g = _grads(stq, at, cu, x, keyvec, bf16, first, dout, grad, plan=plan, stream=side)
    side.synchronize()
    wo, wl, _ = seqref.forward(at, *(y[m] for m in names), S0)
    _within(o.double().cpu().numpy(), wo, _chunk_tol(lens) + _io_step(bf16))
    _within(last.cpu().numpy(), wl, _chunk_tol(lens))
    want = seqref.backward(at, *(y[m] for m in names), S0, do.double().numpy(), dlast)
    for m in names:
        _within(g[m].double().cpu().numpy(), want[m], _grad_tol(m, lens) + _io_step(bf16 and m in "qkv"))
    _within(g["state"].cpu().numpy(), want["state"], _grad_tol("state", lens))


def test_chunk_backward_alone_and_in_a_graph(stq):
    """The same bits alone and in a batch, and at every replay of a captured call."""
    rng = np.random.default_rng(41)
    lens, H, d = [90, 64, 5], 2, 64
    at, cu = _cu(lens)
    x, _ = _inputs(rng, at[-1], H, d, d, True, True)
    do = x["v"] * 0.5
    S0, dl = (torch.from_numpy(rng.normal(size=(3, H, d, d)).astype(np.float32)).cuda() for _ in range(2))
    full = _grads(stq, at, cu, x, True, True, S0, do, dl)
    one = _grads(stq, at[:2], cu[:2], {m: x[m][:90].contiguous() for m in x}, True, True, S0[:1], do[:90].contiguous(),
                 dl[:1])
    for m in full:
        assert torch.equal(one[m], full[m][:len(one[m])]), m
    plan = stq.ChunkPlan(H, d, d, gate=1, max_tokens=at[-1], max_seqs=3, backward=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _grads(stq, at, cu, x, True, True, S0, do, dl, plan)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _grads(stq, at, cu, x, True, True, S0, do, dl, plan)
    for i in range(3):
        new, _ = _inputs(rng, at[-1], H, d, d, True, True)
        for m in x:
            x[m].copy_(new[m])
        want = _grads(stq, at, cu, new, True, True, S0, do, dl)
        graph.replay()
        torch.cuda.synchronize()
        for m in got:
            assert torch.equal(got[m], want[m]), (i, m)


# ------------------------------------------------------------------- verify

def _probs(rng, shape, bf16, hot=2.0):
    x = torch.softmax(torch.from_numpy(rng.normal(size=shape) * hot), -1)
    return x.to(torch.bfloat16 if bf16 else torch.float32)


def _run_verify(stq, tok, lens, p, q, r):
    B, T = tok.shape
    plan = stq.VerifyPlan(B, T, p.shape[2], stq.BF16 if p.dtype == torch.bfloat16 else stq.F32)
    acc = torch.full((B,), -7, dtype=torch.int32, device="cuda")
    nxt = acc.clone()
    stq.verify_draft(plan, _dev(tok, torch.int32), p.cuda(), q.cuda(), _dev(r, torch.float32), acc, nxt,
                     draft_len=None if lens is None else _dev(lens, torch.int32))
    return acc.cpu().numpy(), nxt.cpu().numpy()


@pytest.mark.parametrize("B,T,V,bf16", [(1, 1, 1, False), (5, 3, 7, False), (33, 5, 1000, True), (4, 2, 2048, False),
                                        (7, 4, 2049, True), (3, 70, 50, False), (6, 3, 131073, False)])
def test_verify(stq, B, T, V, bf16):
    rng = np.random.default_rng(B * 1000 + V)
    p, q = _probs(rng, (B, T + 1, V), bf16), _probs(rng, (B, T, V), bf16)
    q = ((q.double() + 3 * p[:, :T].double()) / 4).to(p.dtype)      # mostly agreeing
    tok = rng.integers(0, V, (B, T)).astype(np.int32)
    lens = rng.integers(-1, T + 2, B).astype(np.int32)
    r = rng.uniform(size=(B, T + 1)).astype(np.float32)
    for given in (None, lens):
        acc, nxt = _run_verify(stq, tok, given, p, q, r)
        want = seqref.verify(tok, given, p.double().numpy(), q.double().numpy(), r)
        assert np.array_equal(acc, want[0]) and np.array_equal(nxt, want[1])


def test_verify_edges(stq):
    """Draws of 0 and next to 1, equal rows, one-hot rows, rows of no mass,
    NaN weights, tokens outside the vocabulary, draft probability 0."""
    V, T, B = 300, 2, 9
    p, q = torch.zeros(B, T + 1, V), torch.zeros(B, T, V)
    p[:, :, 10], p[:, :, 200] = 0.25, 0.75
    q[:, :, 10], q[:, :, 200] = 0.75, 0.25
    tok = np.full((B, T), 10, np.int32)
    r = np.full((B, T + 1), 0.5, np.float32)      # 0.5 * 0.75 < 0.25 fails: rejected, rest is 200
    r[1, 0] = np.nextafter(np.float32(1 / 3), np.float32(0))  # just accepted
    r[2, 2] = 0.0
    q[3] = p[3, :T]                                # equal rows: r q < p always holds
    r[3, 2] = np.nextafter(np.float32(1), np.float32(0))
    tok[4] = [-1, 10]
    tok[5] = [V, 10]
    p[6] = 0
    q[7, :, 10] = 0                                # draft probability 0 but target's not: stands
    p[8, 0, 11] = float("nan")
    q[8, 0] = 1.0                                  # nothing left over: p itself, NaN as 0
    acc, nxt = _run_verify(stq, tok, None, p, q, r)
    want = seqref.verify(tok, None, p.double().numpy(), q.double().numpy(), r)
    assert np.array_equal(acc, want[0]) and np.array_equal(nxt, want[1])
    assert list(nxt[:1]) == [200] and nxt[2] == 200 and acc[3] == 2 and nxt[3] == 200
    assert acc[4] == 0 and acc[5] == 0 and nxt[6] == -1 and acc[7] == 2


def test_verify_sampling_without_drafts(stq):
    rng = np.random.default_rng(9)
    p = _probs(rng, (40, 1, 5000), False)
    r = rng.uniform(size=(40, 1)).astype(np.float32)
    tok, q = np.zeros((40, 0), np.int32), p[:, :0]
    acc, nxt = _run_verify(stq, tok, None, p, q, r)
    assert (acc == 0).all()
    c = np.cumsum(p[:, 0].double().numpy(), -1)
    assert np.array_equal(nxt, (c <= r.astype(np.float64) * c[:, -1:]).sum(-1))
