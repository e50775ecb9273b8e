"""What the sequence operators of the library are measured on: the gated delta
rule over whole sequences (``chunk_forward``), its gradients
(``chunk_backward``), the same rule over a few tokens from stored fp32 states
(``recurrent_step``) and the acceptance of drafted tokens (``verify_draft``).

``run`` computes each in its plain form (elementary torch operations) where
``own`` is false, and calls the library where it is true.

Per (sequence, head), with the state S as d_k x d_v:
    S' = diag(a_t) S;  u_t = beta_t (v_t - S'^T k_t);  S = S' + k_t u_t^T;  o_t = S^T q_t.
"""
import math
import random

import torch

own = False

CHUNK = 64          # tokens of one block of the plain chunked form


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the smallest prompt: four requests of 16 tokens, two heads of 64, fp32 inputs (latency)
        _seq("fwd gdn 4x16 f32", "forward", "scalar", "f32", 2, 64, 64, 4, 64, "even", 0),
        # a serving batch of prompts of mixed lengths, GDN layer of 32 heads of 128
        _seq("fwd gdn 24 ragged bf16", "forward", "scalar", "bf16", 32, 128, 128, 24, 24000, "ragged", 1),
        # one long document, KDA layer: few sequences, so the chain of chunks is what counts
        _seq("fwd kda 1x16384 bf16", "forward", "keyvec", "bf16", 16, 128, 128, 1, 16384, "even", 0),
        # a batch of prompts of mixed, odd lengths, KDA layer
        _seq("fwd kda 40 ragged bf16", "forward", "keyvec", "bf16", 32, 128, 128, 40, 16001, "ragged", 2),
        # a small training step, KDA gates, heads with keys of 64 and values of 128
        _seq("bwd kda 3 ragged f32", "backward", "keyvec", "f32", 4, 64, 128, 3, 700, "ragged", 3),
        # a training step: packed documents, GDN layer of 16 heads
        _seq("bwd gdn 8 ragged bf16", "backward", "scalar", "bf16", 16, 128, 128, 8, 16384, "ragged", 4),
        # a training step: four sequences of 2048, KDA layer of 16 heads
        _seq("bwd kda 4x2048 bf16", "backward", "keyvec", "bf16", 16, 128, 128, 4, 8192, "even", 0),
        # one request, one token: latency
        _rec("step gdn 1x1 bf16", "scalar", "bf16", 32, 128, 128, 1, 1),
        # the full serving batch, one token each: the state's bytes
        _rec("step gdn 512x1 bf16", "scalar", "bf16", 32, 128, 128, 512, 1),
        # drafted tokens run ahead: up to six tokens a request, part of them committed
        _rec("step kda 96x6 bf16", "keyvec", "bf16", 32, 128, 128, 96, 6),
        # one request, three drafted tokens, a small vocabulary
        _ver("verify 1x3 V32000", 1, 3, 32000, "f32"),
        # a serving batch with four drafted tokens each and a large odd vocabulary
        _ver("verify 96x4 V129281", 96, 4, 129281, "f32"),
    ]


def draw(rng):
    kind = rng.choice(["forward", "forward", "backward", "step", "verify"])
    if kind == "verify":
        V = _log(rng, 200, 150000)
        T = rng.randint(1, 8)
        B = min(_log(rng, 1, 128), max(1, 60000000 // (V * (2 * T + 1))))
        return _ver(None, B, T, V, rng.choice(["f32", "f32", "bf16"]))
    gate = rng.choice(["scalar", "keyvec"])
    io = rng.choice(["bf16", "bf16", "f32"])
    dk, dv = rng.choice([(128, 128), (128, 128), (64, 64), (64, 128), (128, 64)])
    if kind == "step":
        H, T = rng.choice([1, 2, 4, 8, 16, 32]), rng.choice([1, 1, 2, 3, 5, 8])
        return _rec(None, gate, io, H, dk, dv, min(_log(rng, 1, 500), 16000 // (H * T)), T)
    H = rng.choice([1, 2, 3, 4, 8, 16, 32])
    most = 500000 if kind == "forward" else 120000
    N = _log(rng, 1, min(16384, most // H))
    B = min(N, _log(rng, 1, 48))
    return _seq(None, kind, gate, io, H, dk, dv, B, N, "ragged", rng.randint(1, 1 << 20))


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _seq(name, op, gate, io, H, dk, dv, B, N, mix, mix_seed):
    c = {"op": op, "gate": gate, "io": io, "H": H, "dk": dk, "dv": dv, "B": B, "N": N,
         "lengths": mix, "lengths_seed": mix_seed}
    return dict(c, name=name) if name else c


def _rec(name, gate, io, H, dk, dv, B, T):
    c = {"op": "step", "gate": gate, "io": io, "H": H, "dk": dk, "dv": dv, "B": B, "T": T}
    return dict(c, name=name) if name else c


def _ver(name, B, T, V, io):
    c = {"op": "verify", "B": B, "T": T, "V": V, "io": io}
    return dict(c, name=name) if name else c


def _lengths(case):
    """Lengths of the packed sequences (part of the case: the same for every seed)."""
    B, N = case["B"], case["N"]
    if case["lengths"] == "even":
        return [N // B] * B
    r = random.Random(case["lengths_seed"])
    w = [math.exp(r.gauss(0.0, 0.8)) for _ in range(B)]
    s = sum(w)
    n = [max(1, int(N * x / s)) for x in w]
    while sum(n) > N:
        n[n.index(max(n))] -= 1
    n[n.index(min(n))] += N - sum(n)
    return n


def _step_lengths(case):
    """Tokens per request of a step case: T for the first, then 1..T in turn."""
    return [case["T"] - b % case["T"] for b in range(case["B"])]


# -------------------------------------------------------------------- work

def work(case):
    if case["op"] == "verify":
        e = 4 if case["io"] == "f32" else 2
        B, T, V = case["B"], case["T"], case["V"]
        # one row of each distribution is weighed for the next token
        return {"bytes": float(B * (2 * V * e + T * 16 + 16)), "flops": float(2 * B * V)}
    H, dk, dv = case["H"], case["dk"], case["dv"]
    e = 4 if case["io"] == "f32" else 2
    g = dk if case["gate"] == "keyvec" else 1
    if case["op"] == "step":
        n = sum(_step_lengths(case)) * H
        b = n * ((2 * dk + dv) * e + g * 4 + 4 + dv * 4) + case["B"] * H * dk * dv * 8
        return {"bytes": float(b), "flops": float(n * 6 * dk * dv)}
    n = case["N"] * H
    states = case["B"] * H * dk * dv * 4
    if case["op"] == "forward":
        return {"bytes": float(n * ((2 * dk + 2 * dv) * e + g * 4 + 4) + 2 * states),
                "flops": float(n * 6 * dk * dv)}
    return {"bytes": float(n * ((4 * dk + 3 * dv) * e + 2 * (g * 4 + 4)) + 3 * states),
            "flops": float(n * 18 * dk * dv)}


# ----------------------------------------------------------------- prepare

def _rule_inputs(case, n, gen, dev):
    """q, k of unit length, v normal, gates and write strengths as the layers
    produce them: GDN a = exp(-0.1 softplus(x)), KDA a = 0.8 + 0.2 sigmoid(N(2, 1))."""
    H, dk, dv = case["H"], case["dk"], case["dv"]
    io = torch.float32 if case["io"] == "f32" else torch.bfloat16

    def normal(*shape):
        return torch.randn(*shape, device=dev, generator=gen)

    q, k, v = normal(n, H, dk), normal(n, H, dk), normal(n, H, dv)
    q = (q / q.square().sum(-1, keepdim=True).sqrt()).to(io)
    k = (k / k.square().sum(-1, keepdim=True).sqrt()).to(io)
    v = v.to(io)
    if case["gate"] == "keyvec":
        a = 0.8 + 0.2 * torch.sigmoid(normal(n, H, dk) + 2.0)
    else:
        a = torch.exp(-0.1 * torch.log1p(torch.exp(normal(n, H))))
    beta = torch.sigmoid(normal(n, H))
    return q, k, v, a, beta


def prepare(case, seed):
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    s = {"case": case}
    if case["op"] == "verify":
        B, T, V = case["B"], case["T"], case["V"]
        io = torch.float32 if case["io"] == "f32" else torch.bfloat16
        # a target and a draft that mostly agree, over a long tail of rare tokens
        base = 2.0 * torch.randn(B, T + 1, V, device=dev, generator=gen)
        p = torch.softmax(base, -1)
        q = torch.softmax(base[:, :T] + 0.5 * torch.randn(B, T, V, device=dev, generator=gen), -1)
        del base
        flat = q.reshape(B * T, V).cumsum(-1)
        x = torch.rand(B * T, 1, device=dev, generator=gen) * flat[:, -1:]
        s["draft"] = torch.searchsorted(flat, x).clamp(max=V - 1).reshape(B, T).to(torch.int32)
        s["p"], s["q"] = p.to(io), q.to(io)
        s["len"] = torch.tensor([T - b % (T + 1) if b else T for b in range(B)], dtype=torch.int32, device=dev)
        s["uniform"] = torch.rand(B, T + 1, device=dev, generator=gen)
        if own:
            import linear_attention_recurrent_stq_amd as stq
            s["plan"] = stq.VerifyPlan(B, T, V, stq.F32 if case["io"] == "f32" else stq.BF16)
        return s
    H, dk, dv, B = case["H"], case["dk"], case["dv"], case["B"]
    if case["op"] == "step":
        lens = _step_lengths(case)
    else:
        lens = _lengths(case)
    n = sum(lens)
    s["lens"] = lens
    s["q"], s["k"], s["v"], s["a"], s["beta"] = _rule_inputs(case, n, gen, dev)
    at = [0]
    for x in lens:
        at.append(at[-1] + x)
    s["cu"] = torch.tensor(at, dtype=torch.int32, device=dev)
    s["state"] = 0.1 * torch.randn(B, H, dk, dv, device=dev, generator=gen)
    if case["op"] == "step":
        # requests sit in slots of their own, in another order
        s["slots"] = torch.randperm(B, device=dev, generator=gen).to(torch.int32)
        s["commit"] = torch.tensor([x if case["T"] == 1 else x // 2 for x in lens], dtype=torch.int32, device=dev)
        return s
    if case["op"] == "backward":
        s["do"] = torch.randn(n, H, dv, device=dev, generator=gen).to(s["v"].dtype)
        s["dstate"] = 0.1 * torch.randn(B, H, dk, dv, device=dev, generator=gen)
    if own:
        import linear_attention_recurrent_stq_amd as stq
        s["plan"] = stq.ChunkPlan(H, dk, dv, gate=stq.GATE_KEYVEC if case["gate"] == "keyvec" else stq.GATE_SCALAR,
                                  io_dtype=stq.F32 if case["io"] == "f32" else stq.BF16,
                                  max_tokens=n, max_seqs=B, backward=case["op"] == "backward")
    return s


# --------------------------------------------------------------------- run

def run(s):
    op = s["case"]["op"]
    if own:
        return _run_own(s, op)
    return {"forward": _plain_forward, "backward": _plain_backward, "step": _plain_step,
            "verify": _plain_verify}[op](s)


def _run_own(s, op):
    import linear_attention_recurrent_stq_amd as stq
    if op == "verify":
        B = s["draft"].shape[0]
        n = torch.empty(B, dtype=torch.int32, device="cuda")
        nxt = torch.empty(B, dtype=torch.int32, device="cuda")
        stq.verify_draft(s["plan"], s["draft"], s["p"], s["q"], s["uniform"], n, nxt, draft_len=s["len"])
        return {"accepted": n, "next": nxt}
    q, k, v, a, beta, cu = s["q"], s["k"], s["v"], s["a"], s["beta"], s["cu"]
    if op == "step":
        o = torch.empty(v.shape, dtype=torch.float32, device="cuda")
        stq.recurrent_step(s["state"], s["slots"], cu, q, k, v, a, beta, o, commit=s["commit"])
        return {"o": o, "state": s["state"]}
    if op == "forward":
        o = torch.empty_like(v)
        final = torch.empty_like(s["state"])
        stq.chunk_forward(s["plan"], cu, q, k, v, a, beta, o, initial_state=s["state"], final_state=final)
        return {"o": o, "state": final}
    g = {n: torch.empty_like(x) for n, x in (("q", q), ("k", k), ("v", v), ("a", a), ("beta", beta),
                                             ("state", s["state"]))}
    stq.chunk_backward(s["plan"], cu, q, k, v, a, beta, s["do"], g["q"], g["k"], g["v"], g["a"], g["beta"],
                       initial_state=s["state"], d_final_state=s["dstate"], d_initial_state=g["state"])
    return g


def _pad_index(lens, dev):
    """[B, L] positions of the packed tokens, and a mask of the padding, with L
    a multiple of CHUNK."""
    n = torch.tensor(lens, device=dev)
    first = torch.cumsum(n, 0) - n
    L = -(-max(lens) // CHUNK) * CHUNK
    t = torch.arange(L, device=dev)
    mask = t[None] < n[:, None]
    return torch.where(mask, first[:, None] + t[None], 0), mask


def _padded(s, q, k, v, a, beta):
    """The packed inputs as fp32 [B, L, H, ...]; padding has a = 1 and beta = 0,
    which leaves the state as it is."""
    idx, mask = _pad_index(s["lens"], q.device)
    m3, m2 = mask[:, :, None, None], mask[:, :, None]
    ma = m3 if a.dim() == 3 else m2
    return ((q[idx].float() * m3), (k[idx].float() * m3), (v[idx].float() * m3),
            torch.where(ma, a[idx], 1.0), beta[idx] * m2, idx, mask)


def _plain_chunks(q, k, v, a, beta, S):
    """The chunked form in fp32 on [B, L, H, ...]: every chunk's own products
    at once, then one pass over the chunks for the state."""
    B, L, H, dk = k.shape
    C, n = CHUNK, L // CHUNK

    def chunks(x):
        return x.reshape(B, n, C, H, -1).permute(0, 3, 1, 2, 4).contiguous()

    q, k, v, b = chunks(q), chunks(k), chunks(v), chunks(beta)
    g = torch.cumsum(torch.log(chunks(a)), dim=3)           # [B,H,n,C,dk or 1]
    last = g[:, :, :, -1:]
    kr, qr, kw = k * torch.exp(g), q * torch.exp(g), k * torch.exp(last - g)
    lower = torch.tril(torch.ones(C, C, device=q.device))
    strict = torch.tril(torch.ones(C, C, device=q.device), -1)
    if g.shape[-1] == 1:
        # the difference of sums first, then its exp; above the diagonal it is dropped
        d = torch.exp((g - g.transpose(-1, -2)) * lower) * lower
        kk, qk = k @ k.transpose(-1, -2) * d, q @ k.transpose(-1, -2) * d
    else:
        kd = k * torch.exp(-g)
        kk, qk = kr @ kd.transpose(-1, -2), qr @ kd.transpose(-1, -2)
    A, P = b * kk * strict, qk * lower
    # (I + A)^-1 of a nilpotent A: the product of (I + (-A)^(2^i))
    eye = torch.eye(C, device=q.device)
    X, Y = -A, eye - A
    for _ in range(5):
        X = X @ X
        Y = Y + Y @ X
    Tb = Y * b.transpose(-1, -2)
    U0, W = Tb @ v, Tb @ kr
    dec = torch.exp(last).transpose(-1, -2)                  # [B,H,n,dk or 1,1]
    kwT = kw.transpose(-1, -2).contiguous()
    os = []
    for i in range(n):  # the state passes from chunk to chunk
        u = U0[:, :, i] - W[:, :, i] @ S
        os.append(qr[:, :, i] @ S + P[:, :, i] @ u)
        S = dec[:, :, i] * S + kwT[:, :, i] @ u
    o = torch.stack(os, 2)                                   # [B,H,n,C,dv]
    return o.permute(0, 2, 3, 1, 4).reshape(B, L, H, -1), S


def _plain_forward(s):
    q, k, v, a, beta, idx, mask = _padded(s, s["q"], s["k"], s["v"], s["a"], s["beta"])
    o, S = _plain_chunks(q, k, v, a, beta, s["state"])
    out = torch.empty_like(s["v"])
    out[idx[mask]] = o[mask].to(out.dtype)
    return {"o": out, "state": S}


def _plain_backward(s):
    x = [t.detach().float().requires_grad_() for t in (s["q"], s["k"], s["v"], s["a"], s["beta"], s["state"])]
    with torch.enable_grad():
        q, k, v, a, beta, idx, mask = _padded(s, *x[:5])
        o, S = _plain_chunks(q, k, v, a, beta, x[5])
        do = s["do"][idx].float() * mask[:, :, None, None]
        g = torch.autograd.grad([o, S], x, [do, s["dstate"]])
    like = (s["q"], s["k"], s["v"], s["a"], s["beta"], s["state"])
    return {n: t.to(y.dtype) for n, t, y in zip(("q", "k", "v", "a", "beta", "state"), g, like)}


def _plain_step(s):
    """Token by token: requests with fewer tokens see a = 1, beta = 0 past
    their end."""
    lens, T = s["lens"], max(s["lens"])
    n = torch.tensor(lens, device="cuda")
    first = torch.cumsum(n, 0) - n
    S = s["state"][s["slots"].long()]
    keep = S
    out = torch.empty(s["v"].shape, dtype=torch.float32, device="cuda")
    for t in range(T):
        live = n > t
        at = torch.where(live, first + t, 0)
        q, k, v = s["q"][at].float(), s["k"][at].float(), s["v"][at].float()
        a, beta = s["a"][at], s["beta"][at]
        D = S * (a[..., None] if a.dim() == 3 else a[..., None, None])
        u = beta[..., None] * (v - (D * k[..., None]).sum(-2))
        D = D + k[..., None] * u[..., None, :]
        o = (D * q[..., None]).sum(-2)
        out[torch.where(live, at, first)] = torch.where(live[:, None, None], o, out[first])
        S = torch.where(live[:, None, None, None], D, S)
        keep = torch.where((s["commit"] == t + 1)[:, None, None, None], S, keep)
    s["state"][s["slots"].long()] = keep
    return {"o": out, "state": s["state"]}


def _plain_verify(s):
    p, q, x, r, n = s["p"], s["q"], s["draft"].long(), s["uniform"], s["len"].long()
    B, T = x.shape
    # products and sums in 64 bits: a token at a border is decided the same way everywhere
    px = p[:, :T].gather(-1, x[..., None])[..., 0].double()
    qx = q.gather(-1, x[..., None])[..., 0].double()
    ok = (r[:, :T].double() * qx < px) & (torch.arange(T, device=x.device)[None] < n[:, None])
    acc = torch.cumprod(ok.long(), 1).sum(1)
    rows = torch.arange(B, device=x.device)
    w = p[rows, acc].double()
    rest = (w - q[rows, acc.clamp(max=T - 1)].double()).clamp(min=0.0)
    use = (acc < n) & (rest.sum(-1) > 0)
    w = torch.where(use[:, None], rest, w)
    cum = torch.cumsum(w, -1)
    nxt = (cum <= r[:, T:].double() * cum[:, -1:]).sum(-1)
    return {"accepted": acc.to(torch.int32), "next": nxt.to(torch.int32)}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """The definitions in 64 bits, token by token (verify gives whole numbers alone)."""
    if case["op"] == "verify":
        return None
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    if case["op"] == "step":
        return _exact_step(s)
    if case["op"] == "forward":
        o, S, _ = _exact_run(s)
        return {"o": o, "state": S}
    if case["N"] * case["H"] > 300000:
        return None
    return _exact_backward(s)


def _tok(s, t, names):
    """Token t of every sequence that has one, in 64 bits, and their positions."""
    lens = torch.tensor(s["lens"])
    live = torch.nonzero(lens > t)[:, 0]
    at = (torch.cumsum(lens, 0) - lens + t)[live].cuda()
    return live.cuda(), at, [s[m][at].double() for m in names]


def _col(a):
    return a[..., None] if a.dim() == 3 else a[..., None, None]


def _advance(S, k, v, a, beta):
    D = _col(a) * S
    e = v - torch.einsum("bhij,bhi->bhj", D, k)
    u = beta[..., None] * e
    return D, e, u, D + k[..., :, None] * u[..., None, :]


def _exact_run(s, keep=None):
    """Outputs and last states; the states before the tokens in `keep`."""
    S = s["state"].double()
    o = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
    kept = {}
    for t in range(max(s["lens"])):
        if keep is not None and t in keep:
            kept[t] = S.clone()
        live, at, (q, k, v, a, beta) = _tok(s, t, ("q", "k", "v", "a", "beta"))
        S1 = _advance(S[live], k, v, a, beta)[3]
        o[at] = torch.einsum("bhij,bhi->bhj", S1, q)
        S[live] = S1
    return o, S, kept


def _exact_step(s):
    slots = s["slots"].long()
    S = s["state"][slots].double()
    pool = s["state"].double()
    o = torch.zeros(s["v"].shape, dtype=torch.float64, device="cuda")
    commit = s["commit"].tolist()
    for t in range(max(s["lens"])):
        live, at, (q, k, v, a, beta) = _tok(s, t, ("q", "k", "v", "a", "beta"))
        S1 = _advance(S[live], k, v, a, beta)[3]
        o[at] = torch.einsum("bhij,bhi->bhj", S1, q)
        S[live] = S1
        done = torch.tensor([b for b, c in enumerate(commit) if c == t + 1], device="cuda", dtype=torch.long)
        pool[slots[done]] = S[done]
    return {"o": o, "state": pool}


def _exact_backward(s):
    T, step = max(s["lens"]), 64
    _, _, kept = _exact_run(s, set(range(0, T, step)))
    z = {m: torch.zeros(s[m].shape, dtype=torch.float64, device="cuda") for m in ("q", "k", "v", "a", "beta")}
    dS = s["dstate"].double()
    for t0 in range((T - 1) // step * step, -1, -step):
        S, seen = kept[t0], []
        for t in range(t0, min(T, t0 + step)):
            live, at, x = _tok(s, t, ("q", "k", "v", "a", "beta", "do"))
            D, e, u, S1 = _advance(S[live], *x[1:5])
            seen.append((live, at, x, S[live], D, e, u, S1))
            S = S.clone()
            S[live] = S1
        for live, at, (q, k, v, a, beta, do), S0, D, e, u, S1 in reversed(seen):
            z["q"][at] = torch.einsum("bhij,bhj->bhi", S1, do)
            G = dS[live] + q[..., :, None] * do[..., None, :]
            du = torch.einsum("bhij,bhi->bhj", G, k)
            dk = torch.einsum("bhij,bhj->bhi", G, u)
            z["beta"][at] = (du * e).sum(-1)
            de = beta[..., None] * du
            z["v"][at] = de
            dk -= torch.einsum("bhij,bhj->bhi", D, de)
            z["k"][at] = dk
            G = G - k[..., :, None] * de[..., None, :]
            da = (G * S0).sum(-1)
            z["a"][at] = da if a.dim() == 3 else da.sum(-1)
            dS[live] = _col(a) * G
    return dict(z, state=dS)
