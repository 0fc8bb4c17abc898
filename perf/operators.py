"""Cases for timing and checking the training operators of the memory layer.

Three families: the scaled row lookup and its gradient by sorted ids, the
gated linear recurrence (scan, backward pass, one-token step) and the
distillation loss from a teacher's top logits (with its gradient).

With ``own`` false, ``run`` computes a case from elementary torch operations
in 32 bits, rounded once to the output's type; with ``own`` true it makes the
calls of this package.  ``exact`` gives the same outputs from the definitions
in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
WIDTH = {"bf16": 2, "f32": 4}


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of the generic shape: 32 sequences, 16 rows of 80 each; latency only
        dict(name="lookup-decode", op="lookup", type="bf16", tokens=32, cols=16, dim=80, rows=1_000_003, pad=0.0),
        # the memory of a prefill batch: 24 rows of 256 for each of 16,384 positions
        dict(name="lookup-prefill", op="lookup", type="bf16", tokens=16384, cols=24, dim=256, rows=8_000_000, pad=0.05),
        # the token embedding's gradient: dense over the compressed vocabulary, hidden 5120
        dict(name="grad-dense-vocab", op="grad", type="bf16", tokens=16384, cols=1, dim=5120, rows=99092, pad=0.05),
        # the n-gram table's gradient: 393,216 rows of a 48-million-row table, summed per distinct row
        dict(name="grad-rows-ngram", op="grad_rows", type="bf16", tokens=16384, cols=24, dim=256, rows=48_000_000,
             pad=0.05),
        # a ragged prefill batch at hidden 5120 with carried states and image spans
        dict(name="scan-prefill", op="scan", type="bf16", tokens=16384, dim=5120, seqs=4, state=True, pad=0.05),
        # one long document, an odd number of positions, narrow memory of the generic shape
        dict(name="scan-long", op="scan", type="bf16", tokens=65521, dim=1280, seqs=1, state=False, pad=0.0),
        # a training step's forward and backward at hidden 5120, packed sequences
        dict(name="train-prefill", op="train", type="bf16", tokens=16384, dim=5120, seqs=7, state=False, pad=0.05),
        # a small fine-tuning batch in 32 bits, ragged, states carried from the chunk before
        dict(name="train-small-f32", op="train", type="f32", tokens=1023, dim=1280, seqs=3, state=True, pad=0.0),
        # a decode step of 256 sequences at hidden 5120
        dict(name="step-256", op="step", type="bf16", batch=256, dim=5120),
        # a decode step of a few sequences: launch latency
        dict(name="step-4", op="step", type="bf16", batch=4, dim=1280),
        # a training batch's loss over the raw vocabulary, 64 teacher logits for each position
        dict(name="distill-train", op="distill", type="bf16", tokens=4096, vocab=129280, top=64, tau=2.0, lse=False),
        # a short batch over the compressed vocabulary in 32 bits, the teacher's own normaliser given
        dict(name="distill-small-f32", op="distill", type="f32", tokens=333, vocab=99092, top=20, tau=1.0, lse=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    def width(lo, hi):  # mostly multiples of 8, some odd
        d = spread(lo, hi)
        return d if rng.random() < 0.3 else max(8, d // 8 * 8)

    kind = "f32" if rng.random() < 0.3 else "bf16"
    op = rng.choice(["lookup", "grad", "grad_rows", "scan", "train", "step", "distill"])
    pad = rng.choice([0.0, 0.05, 0.3])
    if op in ("lookup", "grad_rows"):
        cols, dim = rng.choice([1, 3, 16, 24]), width(8, 512)
        tokens = spread(1, max(2, min(65536, 100_000_000 // (cols * dim * WIDTH[kind] // 2))))
        rows = spread(1000, min(48_000_000, 4_000_000_000 // (dim * WIDTH[kind])))
        return dict(op=op, type=kind, tokens=tokens, cols=cols, dim=dim, rows=rows, pad=pad)
    if op == "grad":
        dim = width(64, 5120)
        rows = spread(1000, max(2000, min(129280, 500_000_000 // dim)))
        tokens = spread(1, max(2, min(65536, 80_000_000 // (dim * WIDTH[kind] // 2))))
        return dict(op=op, type=kind, tokens=tokens, cols=1, dim=dim, rows=rows, pad=pad)
    if op in ("scan", "train"):
        dim = width(64, 5120)
        tokens = spread(1, min(65536, 80_000_000 // (dim * WIDTH[kind] // 2)))
        return dict(op=op, type=kind, tokens=tokens, dim=dim, seqs=min(tokens, spread(1, 64)),
                    state=rng.random() < 0.5, pad=pad)
    if op == "step":
        return dict(op=op, type=kind, batch=spread(1, 1024), dim=width(64, 5120))
    vocab = width(1000, 129280)
    return dict(op=op, type=kind, tokens=spread(1, max(2, min(16384, 500_000_000 // (vocab * WIDTH[kind] // 2)))),
                vocab=vocab, top=spread(1, 128), tau=rng.choice([1.0, 2.0, 4.0]), lse=rng.random() < 0.5)


# --------------------------------------------------------------------------- inputs

def _zipf(shape, n, gen):
    """Row numbers with probabilities falling as 1 / rank^1.1, by inverting the continuous law's distribution."""
    u = torch.rand(shape, generator=gen, device=DEV, dtype=torch.float64)
    rank = ((1.0 - u * (1.0 - float(n) ** -0.1)) ** -10.0).floor().clamp_(1, n).long() - 1
    return (rank * 2654435761 + 12345) % n  # frequent rows lie apart, as hashed or unordered ids do


def _normal(shape, kind, gen, scale=1.0):
    return torch.empty(shape, device=DEV, dtype=TYPES[kind]).normal_(0.0, scale, generator=gen)


def _cuts(tokens, seqs, gen):
    """Ragged sequences: [0, cuts..., tokens], none of them empty unless two cuts fall together."""
    inner = torch.randint(0, tokens + 1, (seqs - 1,), generator=gen, device=DEV).sort().values
    edge = torch.zeros(1, dtype=torch.int64, device=DEV)
    return torch.cat([edge, inner, edge + tokens])


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    c = dict(case)
    op, kind = c["op"], c["type"]
    s = dict(case=c, op=op)
    if op in ("lookup", "grad", "grad_rows"):
        T, C, D, R = c["tokens"], c["cols"], c["dim"], c["rows"]
        ids = _zipf((T, C), R, gen)
        pad = torch.rand((T, 1), generator=gen, device=DEV) < c["pad"]  # image positions have no rows
        s["ids"] = torch.where(pad, torch.full_like(ids, -1), ids).to(torch.int32)
        s["scale"] = math.sqrt(D)
        if op == "lookup":
            s["table"] = _normal((R, D), kind, gen, 0.02)
        else:
            s["dout"] = _normal((T, C * D), kind, gen, 0.01)
            s["rows"] = R
    elif op in ("scan", "train"):
        T, D, S = c["tokens"], c["dim"], c["seqs"]
        s["x"] = _normal((T, D), kind, gen)
        s["g"] = _normal((T, D), kind, gen, 1.5).add_(2.0)  # gates around 0.88, some close to one
        s["cu"] = _cuts(T, S, gen)
        s["mask"] = (torch.rand(T, generator=gen, device=DEV) < c["pad"]).to(torch.uint8) if c["pad"] else None
        s["state"] = s["slots"] = s["dstate"] = None
        if c["state"]:
            s["state"] = _normal((S + 2, D), "f32", gen)
            s["slots"] = torch.randperm(S + 2, generator=gen, device=DEV)[:S].to(torch.int32)
        if op == "train":
            s["dy"] = _normal((T, D), kind, gen, 0.1)
            if c["state"]:
                s["dstate"] = _normal((S + 2, D), "f32", gen, 0.1)
    elif op == "step":
        B, D = c["batch"], c["dim"]
        s["x"] = _normal((B, D), kind, gen)
        s["g"] = _normal((B, D), kind, gen, 1.5).add_(2.0)
        s["state"] = _normal((B + 3, D), "f32", gen)
        s["slots"] = torch.randperm(B + 3, generator=gen, device=DEV)[:B].to(torch.int32)
    else:
        T, V, K = c["tokens"], c["vocab"], c["top"]
        z = _normal((T, V), kind, gen, 2.0)
        room = max(1, V // K)  # the K ids of a position are distinct
        ids = torch.arange(K, device=DEV) * room + torch.randint(0, room, (T, K), generator=gen, device=DEV)
        ids = (ids + torch.randint(0, V, (T, 1), generator=gen, device=DEV)) % V
        t = 12.0 - 8.0 * torch.rand((T, K), generator=gen, device=DEV).sort(dim=1).values
        near = (t + torch.randn((T, K), generator=gen, device=DEV)).to(z.dtype)
        z.scatter_(1, ids, near)  # the student agrees with the teacher roughly
        short = torch.rand((T, 1), generator=gen, device=DEV) < 0.1  # some positions have fewer entries, a few none
        keep = torch.randint(0, K + 1, (T, 1), generator=gen, device=DEV)
        drop = short & (torch.arange(K, device=DEV) >= keep)
        s["z"], s["tau"] = z, c["tau"]
        s["ids"] = torch.where(drop, torch.full_like(ids, -1), ids).to(torch.int32)
        s["t"] = t
        s["lse"] = None
        if c["lse"]:  # the teacher's tail holds a tenth to a third of its mass
            top = torch.logsumexp(t.double() / c["tau"], dim=1)
            s["lse"] = (top + 0.1 + 0.3 * torch.rand(T, generator=gen, device=DEV, dtype=torch.float64)).float()
        w = (torch.rand(T, generator=gen, device=DEV) >= 0.05).float() / T  # prompt positions carry no loss
        s["weight"] = w
    return s


# --------------------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import hashed_gram_conditional_gb300 as eg
    op = s["op"]
    if op == "lookup":
        return eg.engram_lookup(s["table"], s["ids"], s["scale"])
    if op == "grad":
        return eg.engram_lookup_grad(s["dout"], s["ids"], s["rows"], s["scale"])
    if op == "grad_rows":
        return eg.engram_lookup_grad_rows(s["dout"], s["ids"], s["rows"], s["scale"])
    if op == "scan":
        y = eg.engram_recurrence(s["x"], s["g"], s["cu"], mask=s["mask"], state=s["state"], slots=s["slots"])
        return [y] if s["state"] is None else [y, s["state"]]  # the states move on, as from chunk to chunk
    if op == "train":
        carry = eg.recurrence_carry(s["x"].shape[0], s["x"].shape[1], s["x"].device)
        out = None if s["state"] is None else torch.clone(s["state"])
        y = eg.engram_recurrence(s["x"], s["g"], s["cu"], mask=s["mask"], state=s["state"], slots=s["slots"],
                                 state_out=out, carry=carry)
        dstate = None if s["dstate"] is None else torch.clone(s["dstate"])
        dx, dg = eg.engram_recurrence_grad(s["dy"], s["x"], s["g"], carry, s["cu"], mask=s["mask"], state=s["state"],
                                           slots=s["slots"], dstate=dstate)
        return [y, dx, dg] if out is None else [y, out, dx, dg, dstate]
    if op == "step":
        y = eg.engram_recurrence_step(s["x"], s["g"], s["slots"], s["state"])
        return [y, s["state"]]
    dz = torch.empty_like(s["z"])
    loss = eg.engram_distill(s["z"], s["ids"], s["t"], temperature=s["tau"], weight=s["weight"],
                             teacher_lse=s["lse"], dlogits=dz)
    return [loss, dz]


def _run_plain(s):
    op = s["op"]
    if op == "lookup":
        return _plain_lookup(s["table"], s["ids"], s["scale"])
    if op == "grad":
        return _plain_grad(s["dout"], s["ids"], s["rows"], s["scale"])
    if op == "grad_rows":
        return _plain_grad_rows(s["dout"], s["ids"], s["rows"], s["scale"])
    if op in ("scan", "train"):
        return _plain_recurrence(s)
    if op == "step":
        return _plain_step(s)
    return _plain_distill(s)


def _plain_lookup(table, ids, scale):
    R, D = table.shape
    ok = (ids >= 0) & (ids < R)
    rows = table[ids.clamp(0, R - 1).long()].float() * scale
    return (rows * ok[..., None]).to(table.dtype).view(ids.shape[0], -1)


def _plain_grad(dout, ids, R, scale):
    n = ids.numel()
    ids = ids.view(-1)
    ok = (ids >= 0) & (ids < R)
    d = dout.view(n, -1).float() * (ok[:, None] * scale)
    return torch.zeros((R, d.shape[1]), device=d.device).index_add_(0, ids.clamp(0, R - 1).long(), d)


def _plain_grad_rows(dout, ids, R, scale):
    n = ids.numel()
    ids = ids.view(-1)
    ok = (ids >= 0) & (ids < R)
    key, order = torch.sort(torch.where(ok, ids, R), stable=True)  # entries without a row go last
    valid = key < R
    first = valid.clone()
    first[1:] &= key[1:] != key[:-1]
    place = (torch.cumsum(first, 0) - 1).clamp_min_(0)  # which distinct row an entry belongs to
    d = dout.view(n, -1)[order].float() * (valid[:, None] * scale)
    grad = torch.zeros_like(d).index_add_(0, place, d)
    rows = torch.full((n + 1,), -1, dtype=torch.int32, device=d.device)
    rows.scatter_(0, torch.where(first, place, n), key.to(torch.int32))
    rows[n] = -1
    return [rows[:n], grad, first.sum().to(torch.int32).view(1)]


def _scan(a, b):
    """s_t = a_t s_{t-1} + b_t from zero, by doubling: after each round a term covers twice as many positions."""
    d, T = 1, a.shape[0]
    while d < T:
        b = torch.cat([b[:d], b[d:] + a[d:] * b[:-d]])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return b


def _plain_recurrence(s):
    x, cu, kind = s["x"].float(), s["cu"], s["x"].dtype
    T = x.shape[0]
    t = torch.arange(T, device=x.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    first = (t == cu[seq])[:, None]
    live = torch.ones_like(first) if s["mask"] is None else (s["mask"] == 0)[:, None]
    f = torch.sigmoid(s["g"].float())
    u = torch.sigmoid(-s["g"].float())
    keep = torch.where(live, f, 1.0)  # a masked position holds the state
    b = torch.where(live, u * x, 0.0)
    s0 = torch.zeros_like(x[:1])
    if s["state"] is not None:
        s0 = s["state"][s["slots"].long()][seq]
    a = torch.where(first, 0.0, keep)
    h = _scan(a, torch.where(first, b + keep * s0, b))
    got = [torch.where(live, h, 0.0).to(kind)]
    some = (cu[1:] > cu[:-1])[:, None]
    last, slots = (cu[1:] - 1).clamp_min(0), None
    if s["state"] is not None:
        slots = s["slots"].long()
        out = s["state"].clone() if s["op"] == "train" else s["state"]
        out[slots] = torch.where(some, h[last], out[slots])
        got.append(out)
    if s["op"] == "scan":
        return got
    dy = torch.where(live, s["dy"].float(), 0.0)
    if s["dstate"] is not None:  # an empty sequence adds nothing, and passes its gradient on
        dy = dy.index_add(0, last, torch.where(some, s["dstate"][slots], 0.0))
    back = torch.cat([a[1:], torch.zeros_like(a[:1])])
    lam = _scan(back.flip(0), dy.flip(0)).flip(0)
    before = torch.where(first, s0, torch.cat([torch.zeros_like(h[:1]), h[:-1]]))
    got.append(torch.where(live, lam * u, 0.0).to(kind))
    got.append(torch.where(live, lam * (before - x) * f * u, 0.0).to(kind))
    if s["dstate"] is not None:
        at = cu[:-1].clamp_max(T - 1)
        ds = s["dstate"].clone()
        ds[slots] = torch.where(some, lam[at] * keep[at], ds[slots])
        got.append(ds)
    return got


def _plain_step(s):
    slots = s["slots"].long()
    g = s["g"].float()
    new = torch.sigmoid(g) * s["state"][slots] + torch.sigmoid(-g) * s["x"].float()
    s["state"][slots] = new
    return [new.to(s["x"].dtype), s["state"]]


def _plain_distill(s):
    tau, V = s["tau"], s["z"].shape[1]
    z = s["z"].float() / tau
    z = z - z.max(dim=1, keepdim=True).values
    lnq = z - torch.log(torch.exp(z).sum(dim=1, keepdim=True))
    ok = (s["ids"] >= 0) & (s["ids"] < V)
    t = torch.where(ok, s["t"] / tau, float("-inf"))
    if s["lse"] is None:
        top = t.max(dim=1, keepdim=True).values
        t = t - torch.where(torch.isfinite(top), top, 0.0)
        lnp = t - torch.log(torch.exp(t).sum(dim=1, keepdim=True).clamp_min(1e-37))
    else:
        lnp = t - s["lse"][:, None]
    p = torch.where(ok, torch.exp(lnp), 0.0)
    ids = s["ids"].clamp(0, V - 1).long()
    term = torch.where(p > 0, p * (lnp - lnq.gather(1, ids)), 0.0)
    loss = s["weight"] * (tau * tau) * term.sum(dim=1)
    dz = torch.exp(lnq) * p.sum(dim=1, keepdim=True)
    dz.scatter_add_(1, ids, -p)
    return [loss, (dz * (s["weight"] * tau)[:, None]).to(s["z"].dtype)]


# --------------------------------------------------------------------------- work of one pass

def work(case):
    c, w = case, WIDTH[case["type"]]
    op = c["op"]
    if op in ("lookup", "grad", "grad_rows"):
        n, D = c["tokens"] * c["cols"], c["dim"]
        if op == "lookup":
            return {"bytes": n * (4 + 2 * w * D), "flops": n * D}
        if op == "grad":
            return {"bytes": n * (4 + w * D) + 4 * c["rows"] * D, "flops": n * D}
        return {"bytes": n * (8 + w * D + 4 * D) + 4, "flops": n * D}
    if op in ("scan", "train"):
        n = c["tokens"] * c["dim"]
        extra = 8 * c["seqs"] * c["dim"] * (2 if op == "train" else 1) if c["state"] else 0
        mask = c["tokens"] if c["pad"] else 0
        if op == "scan":
            return {"bytes": 3 * w * n + extra + mask, "flops": 8 * n}
        return {"bytes": 6 * w * n + extra + mask, "flops": 22 * n}
    if op == "step":
        n = c["batch"] * c["dim"]
        return {"bytes": n * (3 * w + 8) + 4 * c["batch"], "flops": 8 * n}
    T, V, K = c["tokens"], c["vocab"], c["top"]
    return {"bytes": T * (2 * w * V + 8 * K + 8 + (4 if c["lse"] else 0)), "flops": 8 * T * V}


# --------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op == "lookup":
        table, ids = s["table"], s["ids"].view(-1)
        out = torch.zeros((ids.numel(), table.shape[1]), dtype=torch.float64, device=DEV)
        at = torch.nonzero((ids >= 0) & (ids < table.shape[0]))[:, 0]
        out[at] = table[ids[at].long()].double() * s["scale"]
        return out.view(s["ids"].shape[0], -1)
    if op in ("grad", "grad_rows"):
        ids = s["ids"].view(-1).long()
        at = torch.nonzero((ids >= 0) & (ids < s["rows"]))[:, 0]
        d = s["dout"].view(ids.numel(), -1)
        D = d.shape[1]
        if op == "grad":
            out = torch.zeros((s["rows"], D), dtype=torch.float64, device=DEV)
            out.index_add_(0, ids[at], d[at].double())
            return out.mul_(s["scale"])
        uniq, where = torch.unique(ids[at], sorted=True, return_inverse=True)
        n, m = ids.numel(), uniq.numel()
        rows = torch.full((n,), -1, dtype=torch.int32, device=DEV)
        rows[:m] = uniq.to(torch.int32)
        out = torch.zeros((n, D), dtype=torch.float64, device=DEV)
        out.index_add_(0, where, d[at].double())
        return [rows, out.mul_(s["scale"]), torch.tensor([m], dtype=torch.int32, device=DEV)]
    if op in ("scan", "train"):
        return _exact_recurrence(s)
    if op == "step":
        f = 1.0 / (1.0 + torch.exp(-s["g"].double()))
        state = s["state"].double()
        slots = s["slots"].long()
        new = f * state[slots] + (1.0 - f) * s["x"].double()
        state[slots] = new
        return [new, state]
    return _exact_distill(s)


def _exact_recurrence(s):
    """Position by position, as the recurrence is written."""
    x, g, cu = s["x"], s["g"], s["cu"].tolist()
    T, D = x.shape
    live = [True] * T if s["mask"] is None else [m == 0 for m in s["mask"].tolist()]
    slots = None if s["state"] is None else s["slots"].tolist()
    f = 1.0 / (1.0 + torch.exp(-g.double()))
    y = torch.zeros((T, D), dtype=torch.float64, device=DEV)
    train = s["op"] == "train"
    before = torch.zeros((T, D), dtype=torch.float64, device=DEV) if train else None
    state = None if s["state"] is None else s["state"].double()
    xd = x.double()
    for q in range(len(cu) - 1):
        h = torch.zeros(D, dtype=torch.float64, device=DEV) if state is None else state[slots[q]].clone()
        for t in range(cu[q], cu[q + 1]):
            if train:
                before[t] = h
            if live[t]:
                h = torch.lerp(xd[t], h, f[t])
                y[t] = h
        if state is not None:
            state[slots[q]] = h
    got = [y] if state is None else [y, state]
    if not train:
        return got
    dx = torch.zeros((T, D), dtype=torch.float64, device=DEV)
    dg = torch.zeros((T, D), dtype=torch.float64, device=DEV)
    dstate = None if s["dstate"] is None else s["dstate"].double()
    dy = s["dy"].double()
    lam = torch.zeros((T, D), dtype=torch.float64, device=DEV)
    for q in range(len(cu) - 1):
        l = torch.zeros(D, dtype=torch.float64, device=DEV) if dstate is None else dstate[slots[q]].clone()
        for t in range(cu[q + 1] - 1, cu[q] - 1, -1):
            if live[t]:
                l = l + dy[t]
                lam[t] = l
                l = l * f[t]
        if dstate is not None:
            dstate[slots[q]] = l
    dx = lam * (1.0 - f)
    dg = lam * (before - xd) * f * (1.0 - f)
    return got + [dx, dg] + ([] if dstate is None else [dstate])


def _exact_distill(s):
    tau, V = s["tau"], s["z"].shape[1]
    T = s["z"].shape[0]
    step = max(1, 100_000_000 // V)
    dz = torch.empty((T, V), dtype=torch.float64, device=DEV)
    loss = torch.empty(T, dtype=torch.float64, device=DEV)
    for a in range(0, T, step):
        b = min(T, a + step)
        lnq = torch.log_softmax(s["z"][a:b].double() / tau, dim=1)
        ok = (s["ids"][a:b] >= 0) & (s["ids"][a:b] < V)
        t = s["t"][a:b].double() / tau
        norm = torch.logsumexp(t.masked_fill(~ok, -math.inf), dim=1) if s["lse"] is None else s["lse"][a:b].double()
        lnp = t - norm[:, None]
        p = torch.exp(lnp).masked_fill(~ok, 0.0)
        ids = s["ids"][a:b].long().masked_fill(~ok, 0)
        w = s["weight"][a:b].double()
        gap = (lnp - lnq.gather(1, ids)).masked_fill(~ok, 0.0)
        loss[a:b] = w * tau * tau * (p * gap).sum(dim=1)
        dz[a:b] = torch.exp(lnq).mul_(p.sum(dim=1, keepdim=True)).scatter_add_(1, ids, -p).mul_((w * tau)[:, None])
    return [loss, dz]
