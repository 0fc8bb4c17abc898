"""Cases for timing and checking the operators of a gated memory block and of training it on rewards.

Three families: the gated delta rule (a memory that is a matrix for each head:
a whole sequence, its backward pass, one token), the norm behind a block with
its gate, residual scale and the norm in front of the next block (and its
backward pass), and the clipped policy loss with its gradient.

With ``own`` false, ``run`` computes a case from elementary torch operations
in 32 bits (the decays' running sums in 64), rounded once to the output's type;
with ``own`` true it makes the calls of this package.  ``exact`` gives the same
outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
WIDTH = {"bf16": 2, "f32": 4}
EPS = 1e-6
CHUNK = 64  # of the plain form


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # a ragged prefill batch of four sequences, states carried on, image spans; two value heads for a key head
        dict(name="delta-prefill", op="delta", type="bf16", tokens=16384, keys=20, heads=40, dk=128, dv=128, seqs=4,
             state=True, pad=0.05),
        # one long document, an odd number of positions, few heads
        dict(name="delta-long", op="delta", type="bf16", tokens=16381, keys=10, heads=10, dk=128, dv=128, seqs=1,
             state=False, pad=0.0),
        # a training step's forward and backward, packed sequences
        dict(name="delta-train", op="delta_train", type="bf16", tokens=4096, keys=20, heads=40, dk=128, dv=128, seqs=7,
             state=False, pad=0.05),
        # a small fine-tuning batch in 32 bits, odd head widths, states carried from the chunk before
        dict(name="delta-train-small-f32", op="delta_train", type="f32", tokens=509, keys=2, heads=4, dk=80, dv=72,
             seqs=3, state=True, pad=0.0),
        # a decode step of 256 sequences
        dict(name="delta-step-256", op="delta_step", type="bf16", batch=256, keys=20, heads=40, dk=128, dv=128),
        # a decode step of a few sequences: launch latency
        dict(name="delta-step-4", op="delta_step", type="bf16", batch=4, keys=10, heads=10, dk=128, dv=128),
        # between two blocks of a prefill batch at hidden 5120: gate, residual scale and the next block's norm
        dict(name="norm-prefill", op="norm", type="bf16", tokens=16384, dim=5120, groups=1, gate=True, res=True,
             next=True),
        # the heads' outputs of a decode step, normalised and gated
        dict(name="norm-heads-256", op="norm", type="bf16", tokens=256, dim=5120, groups=40, gate=True, res=False,
             next=False),
        # the same place in a training step's backward pass
        dict(name="norm-grad", op="norm_grad", type="bf16", tokens=16384, dim=5120, groups=1, gate=True, res=True,
             next=True),
        # a small fine-tuning batch in 32 bits, odd rows, the norm by heads
        dict(name="norm-grad-small-f32", op="norm_grad", type="f32", tokens=1023, dim=1280, groups=10, gate=True,
             res=True, next=True),
        # a training batch's clipped loss over the raw vocabulary with a KL term
        dict(name="policy-train", op="policy", type="bf16", tokens=4096, vocab=129280, kl=0.05, tau=1.0, old=True),
        # a short batch over the compressed vocabulary in 32 bits, sampled by these very weights
        dict(name="policy-small-f32", op="policy", type="f32", tokens=333, vocab=99092, kl=0.0, tau=0.7, old=False),
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    def width(lo, hi):  # mostly multiples of 8, some odd
        d = spread(lo, hi)
        return d if rng.random() < 0.3 else max(8, d // 8 * 8)

    kind = "f32" if rng.random() < 0.3 else "bf16"
    op = rng.choice(["delta", "delta", "delta_train", "delta_train", "delta_step", "norm", "norm_grad", "policy"])
    if op.startswith("delta"):
        keys, group = spread(1, 20), rng.choice([1, 1, 2, 4])
        dk, dv = rng.choice([64, 128, width(8, 128)]), rng.choice([64, 128, width(8, 128)])
        c = dict(op=op, type=kind, keys=keys, heads=keys * group, dk=dk, dv=dv)
        if op == "delta_step":
            return dict(c, batch=spread(1, max(2, min(1024, 160_000_000 // (keys * group * dk * dv)))))
        most = (100_000_000 if op == "delta" else 20_000_000) // (2 if kind == "f32" else 1)
        tokens = spread(1, min(16384 if op == "delta" else 4096, most // (keys * group * max(dk, dv))))
        return dict(c, tokens=tokens, seqs=min(tokens, spread(1, 64)), state=rng.random() < 0.5,
                    pad=rng.choice([0.0, 0.05, 0.3]))
    if op.startswith("norm"):
        groups = rng.choice([1, 1, 4, 40])
        dim = groups * width(8, max(16, 8192 // groups))
        tokens = spread(1, min(65536, 80_000_000 // (dim * WIDTH[kind] // 2)))
        return dict(op=op, type=kind, tokens=tokens, dim=dim, groups=groups, gate=rng.random() < 0.7,
                    res=rng.random() < 0.7, next=rng.random() < 0.7)
    vocab = width(1000, 129280)
    return dict(op=op, type=kind, tokens=spread(1, max(2, min(16384, 500_000_000 // (vocab * WIDTH[kind] // 2)))),
                vocab=vocab, kl=rng.choice([0.0, 0.05, 0.2]), tau=rng.choice([0.7, 1.0]), old=rng.random() < 0.7)


# --------------------------------------------------------------------------- inputs

def _normal(shape, kind, gen, scale=1.0, shift=0.0):
    return torch.empty(shape, device=DEV, dtype=TYPES[kind]).normal_(shift, scale, generator=gen)


def _unit(rows, heads, d, kind, gen):
    """Rows of unit vectors, one for each head, as a norm in front of the memory leaves them."""
    x = torch.randn((rows, heads, d), generator=gen, device=DEV)
    return (x / x.norm(dim=2, keepdim=True)).to(TYPES[kind]).view(rows, heads * d)


def _cuts(tokens, seqs, rng):
    """Ragged sequences: [0, cuts..., tokens], none of them empty unless two cuts fall together."""
    return [0] + sorted(torch.randint(0, tokens + 1, (seqs - 1,), generator=rng).tolist()) + [tokens]


def _plan(cu):
    """Where the chunks of the plain form lie: positions [n][CHUNK] (-1: none), and the chunks that follow one another."""
    starts, seq_of, rounds = [], [], []
    for q in range(len(cu) - 1):
        for j, t in enumerate(range(cu[q], cu[q + 1], CHUNK)):
            if j == len(rounds):
                rounds.append([])
            rounds[j].append(len(starts))
            starts.append(t)
            seq_of.append(q)
    ends = torch.tensor([cu[q + 1] for q in seq_of], device=DEV)
    at = torch.tensor(starts, device=DEV)[:, None] + torch.arange(CHUNK, device=DEV)
    seq = torch.tensor(seq_of, device=DEV)
    some = torch.tensor([q for q in range(len(cu) - 1) if cu[q + 1] > cu[q]], device=DEV)
    return dict(at=torch.where(at < ends[:, None], at, -1), seq=seq, some=some,
                rounds=[torch.tensor(r, device=DEV) for r in rounds], round_seq=[seq[torch.tensor(r)] for r in rounds])


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    c = dict(case)
    op, kind = c["op"], c["type"]
    s = dict(case=c, op=op)
    if op.startswith("delta"):
        step = op == "delta_step"
        T, Hk, H, dk, dv = c["batch" if step else "tokens"], c["keys"], c["heads"], c["dk"], c["dv"]
        s["keys"], s["scale"] = Hk, dk ** -0.5
        s["q"], s["k"] = _unit(T, Hk, dk, kind, gen), _unit(T, Hk, dk, kind, gen)
        s["v"] = _normal((T, H * dv), kind, gen)
        s["g"] = _normal((T, H), kind, gen, 1.5, 4.0)  # decays around 0.98, some close to one
        s["b"] = _normal((T, H), kind, gen)
        if step:
            s["state"] = _normal((T + 3, H, dk, dv), "f32", gen, 0.3)
            s["slots"] = torch.randperm(T + 3, generator=gen, device=DEV)[:T].to(torch.int32)
            return s
        S = c["seqs"]
        host = torch.Generator()
        host.manual_seed(seed)
        cu = _cuts(T, S, host)
        s["cu"], s["cuts"], s["plan"] = torch.tensor(cu, device=DEV), cu, _plan(cu)
        s["mask"] = (torch.rand(T, generator=gen, device=DEV) < c["pad"]).to(torch.uint8) if c["pad"] else None
        s["state"] = s["slots"] = s["dstate"] = None
        if c["state"]:
            s["state"] = _normal((S + 2, H, dk, dv), "f32", gen, 0.3)
            s["slots"] = torch.randperm(S + 2, generator=gen, device=DEV)[:S].to(torch.int32)
        if op == "delta_train":
            s["dy"] = _normal((T, H * dv), kind, gen, 0.1)
            if c["state"]:
                s["dstate"] = _normal((S + 2, H, dk, dv), "f32", gen, 0.1)
    elif op.startswith("norm"):
        T, D, G = c["tokens"], c["dim"], c["groups"]
        s["groups"] = G
        s["y"] = _normal((T, D), kind, gen, 2.0)
        s["z"] = _normal((T, D), kind, gen) if c["gate"] else None
        s["h"] = _normal((T, D), kind, gen, 3.0) if c["res"] else None
        s["w"] = _normal((D // G,), "f32", gen, 0.2, 1.0)
        s["s"] = _normal((D,), "f32", gen, 0.2, 0.5) if c["res"] else None
        s["wn"] = _normal((D,), "f32", gen, 0.2, 1.0) if c["next"] else None
        if op == "norm_grad":
            s["dh"] = _normal((T, D), kind, gen, 0.1)
            s["dx"] = _normal((T, D), kind, gen, 0.1) if c["next"] else None
            s["out"] = _norm_parts(s)["h"]  # the residual stream, as the forward pass left it
    else:
        T, V, tau = c["tokens"], c["vocab"], c["tau"]
        z = _normal((T, V), kind, gen, 2.0)
        ids = torch.randint(0, V, (T,), generator=gen, device=DEV)
        sure = _normal((T,), "f32", gen, 3.0, 9.0).to(z.dtype)  # a sampled token is mostly a likely one
        z.scatter_(1, ids[:, None], sure[:, None])
        prompt = torch.rand(T, generator=gen, device=DEV) < 0.1  # positions of the prompt have no sampled token
        s["z"], s["tau"], s["kl"], s["clip"] = z, tau, c["kl"], (0.2, 0.28)
        s["ids"] = torch.where(prompt, -1, ids).to(torch.int32)
        s["adv"] = _normal((T,), "f32", gen)
        s["weight"] = torch.full((T,), 1.0 / T, device=DEV)
        logp = _logp(z, ids, tau)
        s["old"] = s["ref"] = None
        if c["old"]:  # the weights have moved on a little since the tokens were sampled
            d = _normal((T,), "f32", gen, 0.2)
            for edge in (math.log(1.0 - s["clip"][0]), math.log(1.0 + s["clip"][1])):
                d = torch.where((d - edge).abs() < 1e-3, edge + 1e-3, d)  # the gradient jumps at the clip's edges
            s["old"] = logp - d
        if c["kl"]:
            s["ref"] = logp + _normal((T,), "f32", gen, 0.3)
    return s


def _logp(z, ids, tau):
    """Log-probabilities of ids under softmax(z / tau)."""
    T, V = z.shape
    out = torch.empty(T, device=z.device)
    step = max(1, 200_000_000 // V)
    for a in range(0, T, step):
        x = z[a:a + step].float() / tau
        out[a:a + step] = x.gather(1, ids[a:a + step, None])[:, 0] - torch.logsumexp(x, dim=1)
    return out


# --------------------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import hashed_gram_conditional_gb300 as eg
    op = s["op"]
    if op == "delta_step":
        y = eg.engram_delta_step(s["q"], s["k"], s["v"], s["g"], s["b"], s["slots"], s["state"], s["keys"])
        return [y, s["state"]]
    if op == "delta":
        y = eg.engram_delta(s["q"], s["k"], s["v"], s["g"], s["b"], s["cu"], s["keys"], mask=s["mask"],
                            state=s["state"], slots=s["slots"])
        return [y] if s["state"] is None else [y, s["state"]]  # the states move on, as from chunk to chunk
    if op == "delta_train":
        T, S = s["q"].shape[0], len(s["cuts"]) - 1
        c = s["case"]
        carry = eg.delta_carry(T, S, c["keys"], c["heads"], c["dk"], c["dv"], s["q"].device)
        out = None if s["state"] is None else torch.clone(s["state"])
        y = eg.engram_delta(s["q"], s["k"], s["v"], s["g"], s["b"], s["cu"], s["keys"], mask=s["mask"],
                            state=s["state"], slots=s["slots"], state_out=out, carry=carry)
        dstate = None if s["dstate"] is None else torch.clone(s["dstate"])
        grads = eg.engram_delta_grad(s["dy"], s["q"], s["k"], s["v"], s["g"], s["b"], carry, s["cu"], s["keys"],
                                     mask=s["mask"], slots=s["slots"], dstate=dstate)
        return [y, *grads] if out is None else [y, out, *grads, dstate]
    if op.startswith("norm"):
        if op == "norm_grad":
            got = eg.engram_norm_add_grad(s["dh"], s["y"], s["w"], gate=s["z"], scale=s["s"], h_out=s["out"], dx=s["dx"],
                                          w_next=s["wn"], groups=s["groups"], residual=s["h"] is not None)
            return [x for x in got if x is not None]  # of y, gate, h, w, scale and w_next
        got = eg.engram_norm_add(s["y"], s["w"], gate=s["z"], h=s["h"], scale=s["s"], w_next=s["wn"], groups=s["groups"])
        return [x for x in got if x is not None]  # the stream and the next block's input
    dz = torch.empty_like(s["z"])
    loss, logp = eg.engram_policy(s["z"], s["ids"], s["adv"], old_logp=s["old"], ref_logp=s["ref"], clip=s["clip"],
                                  kl=s["kl"], temperature=s["tau"], weight=s["weight"], dlogits=dz)
    return [loss, logp, dz]


def _run_plain(s):
    op = s["op"]
    if op == "delta_step":
        return _plain_step(s)
    if op.startswith("delta"):
        return _plain_delta(s)
    if op.startswith("norm"):
        return _plain_norm(s)
    return _plain_policy(s)


def _plain_step(s):
    H = s["g"].shape[1]
    slots = s["slots"].long()
    B, Hk = slots.numel(), s["keys"]
    q = s["q"].float().view(B, Hk, -1).repeat_interleave(H // Hk, 1)
    k = s["k"].float().view(B, Hk, -1).repeat_interleave(H // Hk, 1)
    v = s["v"].float().view(B, H, -1)
    S = s["state"][slots] * torch.sigmoid(s["g"].float())[..., None, None]
    u = torch.sigmoid(s["b"].float())[..., None] * (v - torch.einsum("bhkv,bhk->bhv", S, k))
    S = S + k[..., None] * u[..., None, :]
    s["state"][slots] = S
    y = torch.einsum("bhkv,bhk->bhv", S, q) * s["scale"]
    return [y.reshape(B, -1).to(s["q"].dtype), s["state"]]


def _chunks(x, at, heads):
    """[T][heads*d] -> [chunks][heads][CHUNK][d], zeros where a chunk has no position."""
    T = x.shape[0]
    x = torch.cat([x.float(), torch.zeros_like(x[:1], dtype=torch.float32)])[torch.where(at < 0, T, at)]
    return x.view(at.shape[0], CHUNK, heads, -1).transpose(1, 2).contiguous()


def _rows(x, at, T):
    """The way back: [chunks][heads][CHUNK][d] -> [T][heads*d]."""
    n, H, C, d = x.shape
    out = torch.zeros((T + 1, H * d), device=x.device)
    out[torch.where(at < 0, T, at).view(-1)] = x.transpose(1, 2).reshape(n * C, H * d)
    return out[:T]


def _plain_delta(s):
    """In chunks: with c the decays' running sum, D_ti = exp(c_t - c_i) and A = beta D (K K^T) below the diagonal, the
    writes are U = (I + A)^-1 beta (V - exp(c) K S) and the state moves by exp(c_C - c) K^T U."""
    T, Hk = s["q"].shape[0], s["keys"]
    H, kind = s["g"].shape[1], s["q"].dtype
    r, p, scale = H // Hk, s["plan"], s["scale"]
    at = p["at"]
    live = torch.ones((T, 1), dtype=torch.bool, device=DEV) if s["mask"] is None else (s["mask"] == 0)[:, None]
    q, k = (_chunks(torch.where(live, s[n], 0), at, Hk).repeat_interleave(r, 1) for n in ("q", "k"))
    v = _chunks(torch.where(live, s["v"], 0), at, H)
    logf = torch.where(live, torch.nn.functional.logsigmoid(s["g"].double()), 0.0)
    beta = _chunks(torch.where(live, torch.sigmoid(s["b"].float()), 0.0), at, H)
    pad = torch.cat([logf, torch.zeros_like(logf[:1])])[torch.where(at < 0, T, at)].transpose(1, 2)
    c = pad.cumsum(2)
    D = torch.exp((c[..., :, None] - c[..., None, :]).clamp_max(0.0)).float()
    low = torch.ones((CHUNK, CHUNK), device=DEV).tril()
    c, last = c.float()[..., None], torch.exp(c[..., -1:] - c).float()[..., None]
    into, total = torch.exp(c), torch.exp(c[:, :, -1:])
    kk, qk = k @ k.transpose(2, 3) * D, q @ k.transpose(2, 3) * D * (low * scale)
    N, M = -beta * kk * low.tril(-1), torch.eye(CHUNK, device=DEV)
    for _ in range(6):  # (I + N)(I + N^2)(I + N^4)... = (I - N)^-1
        M = M + N @ M
        N = N @ N
    M = M * beta.transpose(2, 3)
    n, dk, dv = at.shape[0], q.shape[3], v.shape[3]
    first = torch.empty((n, H, dk, dv), device=DEV)
    U = torch.empty_like(v)
    S = torch.zeros((len(s["cuts"]) - 1, H, dk, dv), device=DEV)
    slots = None
    if s["state"] is not None:
        slots = s["slots"].long()
        S = s["state"][slots]
    for j, e in zip(p["rounds"], p["round_seq"]):
        kj, Sj = k[j], S[e]
        u = M[j] @ (v[j] - into[j] * (kj @ Sj))
        first[j], U[j] = Sj, u
        S[e] = total[j] * Sj + kj.transpose(2, 3) @ (last[j] * u)
    got = [torch.where(live, _rows(scale * into * (q @ first) + qk @ U, at, T), 0.0).to(kind)]
    if s["state"] is not None:
        out = s["state"].clone() if s["op"] == "delta_train" else s["state"]
        out[slots] = S
        got.append(out)
    if s["op"] == "delta":
        return got
    do = _chunks(torch.where(live, s["dy"], 0), at, H)
    dS = torch.zeros_like(S) if s["dstate"] is None else s["dstate"][slots]
    after, dV = torch.empty_like(first), torch.empty_like(v)
    for j, e in zip(reversed(p["rounds"]), reversed(p["round_seq"])):
        dSj = dS[e]
        w = M[j].transpose(2, 3) @ (qk[j].transpose(2, 3) @ do[j] + last[j] * (k[j] @ dSj))
        after[j], dV[j] = dSj, w
        dS[e] = total[j] * dSj + q[j].transpose(2, 3) @ (scale * into[j] * do[j]) - k[j].transpose(2, 3) @ (into[j] * w)
    F = scale * D * low * (do @ U.transpose(2, 3))
    E = -D * low.tril(-1) * (dV @ U.transpose(2, 3))
    dq0 = scale * into * (do @ first.transpose(2, 3))
    dk0 = -into * (dV @ first.transpose(2, 3))
    dk1 = last * (U @ after.transpose(2, 3))
    dq = dq0 + F @ k
    dk_ = dk0 + dk1 + E @ k + E.transpose(2, 3) @ k + F.transpose(2, 3) @ q
    reads = (q * dq0).sum(3) + (k * dk0).sum(3)
    writes = (k * dk1).sum(3)
    pairs = (F * (q @ k.transpose(2, 3)) + E * (k @ k.transpose(2, 3))) * low.tril(-1)
    whole = (total * first * after).sum((2, 3))[..., None]
    later = lambda x: x.flip(2).cumsum(2).flip(2)  # noqa: E731
    dlog = later(reads + pairs.sum(3) - pairs.sum(2)) + (writes.cumsum(2) - writes) + whole
    db = (dV * U).sum(3)
    f_off, b_off = torch.sigmoid(-s["g"].float()), torch.sigmoid(-s["b"].float())
    beta_rows = _rows(beta, at, T)
    dg = _rows(dlog[..., None], at, T) * f_off
    db = torch.where(beta_rows > 0, _rows(db[..., None], at, T) / beta_rows, 0.0) * b_off
    sum_heads = lambda x: x.view(n, Hk, r, CHUNK, -1).sum(2)  # noqa: E731
    grads = [_rows(sum_heads(dq), at, T), _rows(sum_heads(dk_), at, T), _rows(dV, at, T), dg, db]
    got += [torch.where(live, x, 0.0).to(kind) for x in grads]
    if s["dstate"] is not None:
        ds = s["dstate"].clone()
        ds[slots] = dS
        got.append(ds)
    return got


def _norm_parts(s):
    y, G = s["y"].float(), s["groups"]
    T, D = y.shape
    yg = y.view(T, G, D // G)
    r = torch.rsqrt((yg * yg).mean(2, keepdim=True) + EPS)
    hat = yg * r
    n = (hat * s["w"]).reshape(T, D)
    sz = None if s["z"] is None else torch.sigmoid(s["z"].float())
    act = None if sz is None else s["z"].float() * sz
    o = n if act is None else n * act
    so = o if s["s"] is None else o * s["s"]
    h = (so if s["h"] is None else s["h"].float() + so).to(s["y"].dtype)
    return dict(r=r, hat=hat, n=n, sz=sz, act=act, o=o, h=h)


def _plain_norm(s):
    kind = s["y"].dtype
    p = _norm_parts(s)
    h = s["out"].float() if s["op"] == "norm_grad" else p["h"].float()
    if s["wn"] is not None:
        r2 = torch.rsqrt((h * h).mean(1, keepdim=True) + EPS)
        hhat = h * r2
    if s["op"] == "norm":
        return [p["h"]] + ([] if s["wn"] is None else [(hhat * s["wn"]).to(kind)])
    T, D = h.shape
    dh, dwn = s["dh"].float(), None
    if s["wn"] is not None:
        dx = s["dx"].float()
        dwn = (dx * hhat).sum(0)
        dx = dx * s["wn"]
        dh = dh + r2 * (dx - hhat * (dx * hhat).mean(1, keepdim=True))
    do = dh if s["s"] is None else dh * s["s"]
    dz = None if p["sz"] is None else do * p["n"] * p["sz"] * (1.0 + s["z"].float() * (1.0 - p["sz"]))
    dn = (do if p["act"] is None else do * p["act"]).view(T, s["groups"], -1)
    dw = (dn * p["hat"]).sum((0, 1))
    dn = dn * s["w"]
    dy = p["r"] * (dn - p["hat"] * (dn * p["hat"]).mean(2, keepdim=True))
    out = [dy.reshape(T, D).to(kind)] + ([] if dz is None else [dz.to(kind)])
    out += ([] if s["h"] is None else [dh.to(kind)]) + [dw]
    out += [] if s["s"] is None else [(dh * p["o"]).sum(0)]
    return out + ([] if dwn is None else [dwn])


def _plain_policy(s):
    tau, V = s["tau"], s["z"].shape[1]
    z = s["z"].float() / tau
    z = z - z.max(dim=1, keepdim=True).values
    lnq = z - torch.log(torch.exp(z).sum(dim=1, keepdim=True))
    ok = (s["ids"] >= 0) & (s["ids"] < V)
    ids = s["ids"].clamp(0, V - 1).long()[:, None]
    logp = torch.where(ok, lnq.gather(1, ids)[:, 0], 0.0)
    A = s["adv"]
    r = torch.ones_like(logp) if s["old"] is None else torch.exp(logp - s["old"])
    kept = r * A <= r.clamp(1.0 - s["clip"][0], 1.0 + s["clip"][1]) * A
    loss = -torch.minimum(r * A, r.clamp(1.0 - s["clip"][0], 1.0 + s["clip"][1]) * A)
    d = torch.where(kept, -r * A, 0.0)
    if s["ref"] is not None:
        gap = s["ref"] - logp
        loss = loss + s["kl"] * (torch.expm1(gap) - gap)
        d = d - s["kl"] * torch.expm1(gap)
    w = torch.where(ok, s["weight"], 0.0)
    d = w * d / tau
    dz = torch.exp(lnq) * -d[:, None]
    dz.scatter_add_(1, ids, d[:, None])
    return [w * loss, logp, dz.to(s["z"].dtype)]


# --------------------------------------------------------------------------- work of one pass

def work(case):
    c, w = case, WIDTH[case["type"]]
    op = c["op"]
    if op.startswith("delta"):
        Hk, H, dk, dv = c["keys"], c["heads"], c["dk"], c["dv"]
        T = c["batch"] if op == "delta_step" else c["tokens"]
        row = w * (2 * Hk * dk + 2 * H * dv + 2 * H)
        if op == "delta_step":
            return {"bytes": T * (row + 8 * H * dk * dv + 4), "flops": 7 * T * H * dk * dv}
        mask = T if c["pad"] else 0
        states = 8 * c["seqs"] * H * dk * dv if c["state"] else 0
        if op == "delta":
            return {"bytes": T * row + mask + states, "flops": 7 * T * H * dk * dv}
        back = w * (4 * Hk * dk + 3 * H * dv + 4 * H)  # q, k, v, g, b and dy in, their gradients out
        return {"bytes": T * (row + w * H * dv + back) + mask + 2 * states, "flops": 21 * T * H * dk * dv}
    if op.startswith("norm"):
        n = c["tokens"] * c["dim"] * w
        arrays = 2 + c["gate"] + c["res"] + c["next"]
        if op == "norm":
            return {"bytes": n * arrays, "flops": 12 * c["tokens"] * c["dim"]}
        # dh, y, the gate, and where there is a next norm h and dx in; the gradients of y, the gate and h out
        arrays = 3 + 2 * c["gate"] + c["res"] + 2 * c["next"]
        return {"bytes": n * arrays, "flops": 28 * c["tokens"] * c["dim"]}
    T, V = c["tokens"], c["vocab"]
    return {"bytes": T * (2 * w * V + 20 + (4 if c["old"] else 0) + (4 if c["kl"] else 0)), "flops": 8 * T * V}


# --------------------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op.startswith("delta"):
        return _exact_delta(s)
    if op.startswith("norm"):
        return _exact_norm(s)
    return _exact_policy(s)


def _exact_delta(s):
    """Token by token: S <- f S, u = beta (v - S^T k), S <- S + k u^T, y = scale S^T q."""
    step, train = s["op"] == "delta_step", s["op"] == "delta_train"
    Hk, H = s["keys"], s["g"].shape[1]
    T = s["q"].shape[0]
    q, k = (s[n].double().view(T, Hk, -1).repeat_interleave(H // Hk, 1) for n in ("q", "k"))
    v = s["v"].double().view(T, H, -1)
    f, beta = torch.sigmoid(s["g"].double()), torch.sigmoid(s["b"].double())
    dk, dv, scale = q.shape[2], v.shape[2], s["scale"]
    if step:
        state, slots = s["state"].double(), s["slots"].long()
        S = state[slots] * f[..., None, None]
        u = beta[..., None] * (v - (S * k[..., None]).sum(2))
        S = S + k[..., None] * u[..., None, :]
        state[slots] = S
        return [(scale * (S * q[..., None]).sum(2)).view(T, -1), state]
    live = [True] * T if s["mask"] is None else [m == 0 for m in s["mask"].tolist()]
    cu = s["cuts"]
    slots = None if s["slots"] is None else s["slots"].tolist()
    state = None if s["state"] is None else s["state"].double()
    y = torch.zeros((T, H, dv), dtype=torch.float64, device=DEV)
    before = torch.empty((T, H, dk, dv), dtype=torch.float64, device=DEV) if train else None
    us = torch.zeros((T, H, dv), dtype=torch.float64, device=DEV)
    for n in range(len(cu) - 1):
        S = torch.zeros((H, dk, dv), dtype=torch.float64, device=DEV) if state is None else state[slots[n]].clone()
        for t in range(cu[n], cu[n + 1]):
            if not live[t]:
                continue
            if train:
                before[t] = S
            S = S * f[t][:, None, None]
            u = torch.baddbmm(v[t][:, None], k[t][:, None], S, alpha=-1.0) * beta[t][:, None, None]
            S = torch.baddbmm(S, k[t][:, :, None], u)
            us[t] = u[:, 0]
            y[t] = torch.bmm(q[t][:, None], S)[:, 0]
        if state is not None:
            state[slots[n]] = S
    got = [(y * scale).view(T, -1)] + ([] if state is None else [state])
    if not train:
        return got
    do = s["dy"].double().view(T, H, dv) * scale
    dstate = None if s["dstate"] is None else s["dstate"].double()
    dq, dk_ = torch.zeros_like(q), torch.zeros_like(k)
    dvs, dg, db = torch.zeros_like(v), torch.zeros_like(f), torch.zeros_like(beta)
    for n in range(len(cu) - 1):
        dS = torch.zeros((H, dk, dv), dtype=torch.float64, device=DEV) if dstate is None else dstate[slots[n]].clone()
        for t in range(cu[n + 1] - 1, cu[n] - 1, -1):
            if not live[t]:
                continue
            S = before[t] * f[t][:, None, None]  # after the decay
            after = torch.baddbmm(S, k[t][:, :, None], us[t][:, None])
            dq[t] = torch.bmm(after, do[t][:, :, None])[:, :, 0]
            dS = torch.baddbmm(dS, q[t][:, :, None], do[t][:, None])
            du = torch.bmm(k[t][:, None], dS)[:, 0]
            dvs[t] = beta[t][:, None] * du
            seen = torch.bmm(k[t][:, None], S)[:, 0]
            db[t] = (du * (v[t] - seen)).sum(1) * beta[t] * (1.0 - beta[t])
            dk_[t] = torch.bmm(dS, us[t][:, :, None])[:, :, 0] - torch.bmm(S, dvs[t][:, :, None])[:, :, 0]
            dS = torch.baddbmm(dS, k[t][:, :, None], dvs[t][:, None], alpha=-1.0)
            dg[t] = (dS * S).sum((1, 2)) * (1.0 - f[t])
            dS = dS * f[t][:, None, None]
        if dstate is not None:
            dstate[slots[n]] = dS
    shared = lambda x: x.view(T, Hk, H // Hk, dk).sum(2).view(T, -1)  # noqa: E731
    return got + [shared(dq), shared(dk_), dvs.view(T, -1), dg, db] + ([] if dstate is None else [dstate])


def _exact_norm(s):
    y = s["y"].double()
    T, D = y.shape
    G = s["groups"]
    r1 = ((y.view(T, G, -1) ** 2).mean(2) + EPS) ** -0.5
    r1 = r1.repeat_interleave(D // G, 1)
    w = s["w"].double().repeat(G)
    scale = torch.ones(D, dtype=torch.float64, device=DEV) if s["s"] is None else s["s"].double()
    z = None if s["z"] is None else s["z"].double()
    sig = 1.0 if z is None else 1.0 / (1.0 + torch.exp(-z))
    act = 1.0 if z is None else z * sig
    o = y * r1 * w * act
    h = o * scale + (0.0 if s["h"] is None else s["h"].double())
    out = [h] if s["op"] == "norm" else []
    # the next norm reads the residual stream as it is kept
    hs = (s["out"] if s["op"] == "norm_grad" else h.to(s["y"].dtype)).double()
    r2 = ((hs ** 2).mean(1, keepdim=True) + EPS) ** -0.5
    if s["op"] == "norm":
        return out + ([] if s["wn"] is None else [hs * r2 * s["wn"].double()])
    dh, dwn = s["dh"].double(), None
    if s["wn"] is not None:
        dx = s["dx"].double()
        dwn = (dx * hs * r2).sum(0)
        a = dx * s["wn"].double()
        dh = dh + r2 * a - hs * r2 ** 3 * (a * hs).mean(1, keepdim=True)
    do = dh * scale
    a = do * act * w
    along = (a * y).view(T, G, -1).mean(2).repeat_interleave(D // G, 1)
    out.append(a * r1 - y * r1 ** 3 * along)
    if z is not None:
        out.append(do * y * r1 * w * (sig + z * sig * (1.0 - sig)))
    if s["h"] is not None:
        out.append(dh)
    out.append((do * act * y * r1).view(T, G, -1).sum((0, 1)))
    if s["s"] is not None:
        out.append((dh * o).sum(0))
    return out + ([] if dwn is None else [dwn])


def _exact_policy(s):
    tau, V = s["tau"], s["z"].shape[1]
    T = s["z"].shape[0]
    lo, hi = 1.0 - s["clip"][0], 1.0 + s["clip"][1]
    dz = torch.empty((T, V), dtype=torch.float64, device=DEV)
    loss = torch.zeros(T, dtype=torch.float64, device=DEV)
    logp = torch.zeros(T, dtype=torch.float64, device=DEV)
    step = max(1, 100_000_000 // V)
    for a in range(0, T, step):
        b = min(T, a + step)
        lnq = torch.log_softmax(s["z"][a:b].double() / tau, dim=1)
        ids = s["ids"][a:b].long()
        ok = (ids >= 0) & (ids < V)
        ids = ids.masked_fill(~ok, 0)[:, None]
        lp = lnq.gather(1, ids)[:, 0].masked_fill(~ok, 0.0)
        A, w = s["adv"][a:b].double(), s["weight"][a:b].double().masked_fill(~ok, 0.0)
        r = torch.ones_like(lp) if s["old"] is None else torch.exp(lp - s["old"][a:b].double())
        cut = r.clamp(lo, hi)
        term = -torch.minimum(r * A, cut * A)
        d = torch.where(r * A <= cut * A, -r * A, 0.0)
        if s["ref"] is not None:
            gap = s["ref"][a:b].double() - lp
            term = term + s["kl"] * (torch.exp(gap) - 1.0 - gap)
            d = d + s["kl"] * (1.0 - torch.exp(gap))
        loss[a:b], logp[a:b] = w * term, lp
        d = (w * d / tau)[:, None]
        dz[a:b] = torch.exp(lnq).mul_(-d).scatter_add_(1, ids, d)
    return [loss, logp, dz]
