"""Measured cases of the operators on a language model's logits over the packed token
streams: log probabilities of the streams' tokens (with entropy, log-sum-exp and top
alternatives), distillation from a teacher's top list, and the gradient of each.

Logits are [S, V] (the text stream) or [S, n, V] (n audio streams). With c = scale:

    lse = ln sum_i exp(c x_i)      logprob = c x_token - lse      entropy = -sum_i p_i ln p_i
    d x_i = c (a ([i = token] - p_i) + z p_i - b p_i (ln p_i + entropy))

for upstream gradients a, b, z of logprob, entropy and lse; and for a teacher's list
(id_j, t_j), an id below zero being an empty place,

    q = softmax(t), or with the tail q_j = exp(t_j) and q_r = max(0, 1 - sum q_j)
    loss = sum_j q_j (ln q_j - logprob(id_j)) [+ q_r (ln q_r - ln p_rest)]
    d x_i = g c (Q p_i - sum_{j: id_j = i} q_j) [- g c q_r softmax_rest(x)_i], Q = sum q [+ q_r].
"""
import math

import torch

own = False

TEXT_CARD, AUDIO_CARD, STREAMS = 32000, 2048, 17
ABSENT_EVERY = 50  # one step in 50 has no target or teacher (a pad)


def _case(name, op, S, n, V, dtype, k, tail=False, scale=1.0, streams_major=False):
    c = {"op": op, "S": S, "n": n, "V": V, "dtype": dtype, "k": k, "tail": tail, "scale": scale,
         "streams_major": streams_major}
    return c if name is None else {"name": name, **c}


def listed():
    return [
        # one user's text step: the reply's log probability and 20 alternatives
        _case("logprob text step", "logprob", 1, 0, TEXT_CARD, "bf16", 20),
        # one 80 ms frame of 16 users: 8 audio streams each, sampled at temperature 0.8
        _case("logprob audio step", "logprob", 16, 8, AUDIO_CARD, "bf16", 8, scale=1.25),
        # five minutes of text scored in float32; the pad is a class of its own, so rows are odd
        _case("logprob text 5 min", "logprob", 3750, 0, TEXT_CARD + 1, "f32", 5),
        # scoring a data set's audio streams of both speakers
        _case("logprob audio bulk", "logprob", 16384, 16, AUDIO_CARD, "bf16", 0),
        # policy-gradient step on five minutes of text, with an entropy bonus
        _case("logprob grad text", "logprob_grad", 3750, 0, TEXT_CARD, "bf16", 0),
        # audio heads that were computed one stream after another, float32
        _case("logprob grad audio", "logprob_grad", 3750, 16, AUDIO_CARD, "f32", 0,
              streams_major=True),
        # a short clip with the pad as a class: odd rows
        _case("logprob grad clip", "logprob_grad", 250, 0, TEXT_CARD + 1, "bf16", 0),
        # validation loss of a student against the teacher's 64 best and their tail
        _case("distill text", "distill", 1024, 0, TEXT_CARD, "bf16", 64, tail=True),
        # the same for the audio streams, renormalised, float32
        _case("distill audio", "distill", 3750, 8, AUDIO_CARD, "f32", 20),
        # the training step on five minutes of text
        _case("distill grad text", "distill_grad", 3750, 0, TEXT_CARD, "bf16", 64, tail=True),
        # a large batch of audio frames, softened by a temperature of 2
        _case("distill grad audio", "distill_grad", 16384, 8, AUDIO_CARD, "bf16", 16, scale=0.5),
        # few rows of a large vocabulary
        _case("distill grad long rows", "distill_grad", 100, 0, 131072, "f32", 128, tail=True),
    ]


def draw(rng):
    op = rng.choice(["logprob", "logprob_grad", "distill", "distill_grad"])
    V = int(round(math.exp(rng.uniform(math.log(200), math.log(160000)))))
    n = rng.choice([0, 1, 7, 8, 16]) if V <= 4200 else 0
    most = 120e6
    rows = math.exp(rng.uniform(0.0, math.log(most / V)))
    S = max(1, min(16384, int(rows / max(1, n))))
    dtype = rng.choice(["bf16", "bf16", "f32"])
    k = rng.choice([0, 1, 5, 8, 20, 33, 64]) if op == "logprob" else 0
    if op.startswith("distill"):
        k = int(round(math.exp(rng.uniform(0.0, math.log(128)))))
    return _case(None, op, S, n, V, dtype, k, tail=op.startswith("distill") and rng.random() < 0.5,
                 scale=rng.choice([1.0, 1.0, 0.5, 1.25]),
                 streams_major=n > 1 and rng.random() < 0.5)


def _absent(S):
    return len(range(ABSENT_EVERY - 1, S, ABSENT_EVERY))


def work(case):
    S, n, V, k = case["S"], max(1, case["n"]), case["V"], case["k"]
    size = 2 if case["dtype"] == "bf16" else 4
    rows = S * n
    live = (S - _absent(S)) * n  # rows that have a teacher: the others' loss is 0
    if case["op"] == "logprob":  # entropy and alternatives are those of every row
        return {"bytes": rows * (V * size + 4 + 12 + 8 * k), "flops": 6 * rows * V}
    if case["op"] == "logprob_grad":
        return {"bytes": rows * (2 * V * size + 4 + 8 + 8), "flops": 10 * rows * V}
    lists = rows * k * 8
    if case["op"] == "distill":
        return {"bytes": live * V * size + lists + rows * 4, "flops": 4 * live * V}
    return {"bytes": live * V * size + rows * V * size + lists + rows * 8, "flops": 8 * live * V}


def _logits(case, g):
    """Logits as a model gives them: a normal bulk and a few tokens that stand out."""
    S, n, V = case["S"], max(1, case["n"]), case["V"]
    rows = S * n
    x = torch.empty((rows, V), device="cuda").normal_(0.0, 1.5, generator=g)
    best = torch.randint(0, V, (rows, 12), device="cuda", generator=g)
    lift = torch.empty((rows, 12), device="cuda").uniform_(2.0, 12.0, generator=g)
    x.scatter_add_(1, best, lift)
    return x, best


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    S, n, V, k = case["S"], max(1, case["n"]), case["V"], case["k"]
    dtype = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    x, best = _logits(case, g)
    absent = torch.zeros(S, dtype=torch.bool, device="cuda")
    absent[ABSENT_EVERY - 1::ABSENT_EVERY] = True
    st = {"op": case["op"], "scale": case["scale"], "pad": V, "k": k, "tail": case["tail"]}
    if case["op"].startswith("distill"):
        # the teacher: near the student, its best k as logits, or as log probabilities
        t = x + torch.empty_like(x).normal_(0.0, 0.7, generator=g)
        values, ids = torch.topk(t, min(k, V), dim=1)
        if case["tail"]:
            values = values - torch.logsumexp(t, dim=1, keepdim=True)
        del t
        short = min(k, V) < k
        if short:
            more = (values.shape[0], k - values.shape[1])
            values = torch.cat([values, torch.zeros(more, device="cuda")], 1)
            ids = torch.cat([ids, torch.full(more, -1, device="cuda")], 1)
        ids = ids.to(torch.int32).view(S, n, k).clone()
        ids[absent] = -1
        st["ids"] = ids if case["n"] else ids.view(S, k)
        st["teacher"] = values.view(st["ids"].shape).contiguous()
        st["g"] = torch.full((S, n) if case["n"] else (S,), 1.0 / max(1, (S - _absent(S)) * n),
                             device="cuda")
    else:
        if case["op"] == "logprob":  # tokens that the application does not allow
            x[:, V // 2:V // 2 + V // 100] = -math.inf
        pick = torch.randint(0, 12, (S * n, 1), device="cuda", generator=g)
        token = best.gather(1, pick).to(torch.int32).view(S, n)
        if case["op"] == "logprob":  # a token that was answered is an allowed one
            barred = (token >= V // 2) & (token < V // 2 + V // 100)
            token = torch.where(barred, token - V // 100, token)
        token[absent] = V
        col0 = 1 if case["n"] else 0
        packed = torch.randint(0, V, (S, STREAMS), device="cuda", generator=g, dtype=torch.int32)
        packed[:, col0:col0 + n] = token
        st["tokens"] = packed[:, 1:1 + n] if case["n"] else packed[:, 0]
        adv = torch.empty((S, n), device="cuda").normal_(0.0, 1.0, generator=g) / (S * n)
        bonus = torch.full((S, n), 0.01 / (S * n), device="cuda")
        adv[absent] = 0.0
        bonus[absent] = 0.0
        st["g_logprob"] = adv if case["n"] else adv.view(S)
        st["g_entropy"] = bonus if case["n"] else bonus.view(S)
    x = x.to(dtype)
    if not case["n"]:
        st["logits"] = x
    elif case["streams_major"]:
        st["logits"] = x.view(S, n, V).permute(1, 0, 2).contiguous().permute(1, 0, 2)
    else:
        st["logits"] = x.view(S, n, V)
    return st


# ------------------------------------------------------------------ plain form


def _lse(y):
    m = y.amax(-1, keepdim=True)
    return m + (y - m).exp().sum(-1, keepdim=True).log()


def _top(x, k):
    """The k largest, ties to the lowest index: keys of the value's order, then the index."""
    V = x.shape[-1]
    bits = (x + 0.0).view(torch.int32)
    order = torch.where(bits >= 0, bits, bits ^ 0x7FFFFFFF).long()
    index = torch.arange(V - 1, -1, -1, device=x.device)
    keys = torch.topk((order << 32) | index, min(k, V), dim=-1).values
    return V - 1 - (keys & 0xFFFFFFFF)


def _plain_logprob(st):
    x = st["logits"].float()
    V = x.shape[-1]
    y = x * st["scale"]
    lse = _lse(y)
    tok = st["tokens"].long()
    there = (tok >= 0) & (tok < V) & (tok != st["pad"])
    at = torch.where(there, tok, 0).unsqueeze(-1)
    logp = y - lse
    logprob = torch.where(there, logp.gather(-1, at).squeeze(-1), 0.0)
    p = logp.exp()
    entropy = -(p * torch.where(p > 0, logp, 0.0)).sum(-1)
    return x, logp, p, at, there, logprob, entropy, lse.squeeze(-1)


def _plain_run_logprob(st):
    x, logp, _, _, _, logprob, entropy, lse = _plain_logprob(st)
    out = {"logprob": logprob, "entropy": entropy, "lse": lse}
    if st["k"]:
        ids = _top(x, st["k"])
        out["top_logprob"] = logp.gather(-1, ids)
        out["top_ids"] = ids.to(torch.int32)
    return out


def _plain_run_logprob_grad(st):
    _, logp, p, at, there, logprob, entropy, _ = _plain_logprob(st)
    a = torch.where(there, st["g_logprob"], 0.0).unsqueeze(-1)
    b = st["g_entropy"].unsqueeze(-1)
    d = -p * (a + b * (torch.where(p > 0, logp, 0.0) + entropy.unsqueeze(-1)))
    d.scatter_add_(-1, at, a)
    return {"dlogits": (d * st["scale"]).to(st["logits"].dtype), "logprob": logprob,
            "entropy": entropy}


def _plain_distill(st):
    y = st["logits"].float() * st["scale"]
    logp = y - _lse(y)
    there = st["ids"] >= 0
    at = torch.where(there, st["ids"], 0).long()
    t = torch.where(there, st["teacher"].float(), -math.inf)
    row = there.any(-1, keepdim=True)
    lp = logp.gather(-1, at)
    if not st["tail"]:
        lq = t - torch.where(row, _lse(torch.where(row, t, 0.0)), 0.0)
        q = lq.exp()
        loss = torch.where(q > 0, q * (lq - lp), 0.0).sum(-1)
        return y, logp, at, there, q, loss, None, None
    q64 = t.double().exp()
    q = q64.float()
    qr = torch.where(row, (1.0 - q64.sum(-1, keepdim=True)).clamp_min(0.0), 0.0).float()
    listed_ = torch.zeros_like(y).scatter_add_(-1, at, there.float()) > 0
    rest = torch.where(listed_, -math.inf, y)
    lse_rest = _lse(rest)
    lp_rest = lse_rest - _lse(y)
    loss = torch.where(q > 0, q * (t - lp), 0.0).sum(-1)
    loss = loss + torch.where(qr > 0, qr * (qr.log() - lp_rest), 0.0).squeeze(-1)
    return y, logp, at, there, q, loss, qr, (rest - lse_rest).exp()


def _plain_run_distill(st):
    return {"loss": _plain_distill(st)[5]}


def _plain_run_distill_grad(st):
    _, logp, at, there, q, loss, qr, rest = _plain_distill(st)
    Q = q.sum(-1, keepdim=True)
    d = logp.exp() * (Q if qr is None else Q + qr)
    d.scatter_add_(-1, at, -q)
    if qr is not None:
        d -= qr * rest
    d *= st["g"].unsqueeze(-1) * st["scale"]
    return {"dlogits": d.to(st["logits"].dtype), "loss": loss}


# ------------------------------------------------------------------ the framework's calls


def _own_run(st):
    import split_residual_vector_b200 as mimi

    x, op = st["logits"], st["op"]
    if op == "logprob":
        r = mimi.token_logprobs(x, st["tokens"], pad=st["pad"], scale=st["scale"], top_k=st["k"])
        out = {"logprob": r.logprob, "entropy": r.entropy, "lse": r.lse}
        if st["k"]:
            out["top_logprob"], out["top_ids"] = r.top_logprob, r.top_ids
        return out
    if op == "logprob_grad":
        d, r = mimi.token_logprobs_grad(x, st["tokens"], st["g_logprob"], st["g_entropy"],
                                        pad=st["pad"], scale=st["scale"], values=True)
        return {"dlogits": d, "logprob": r.logprob, "entropy": r.entropy}
    if op == "distill":
        return {"loss": mimi.distill_topk(x, st["ids"], st["teacher"], tail=st["tail"],
                                          scale=st["scale"])}
    d, loss = mimi.distill_topk_grad(x, st["ids"], st["teacher"], st["g"], tail=st["tail"],
                                     scale=st["scale"], loss=True)
    return {"dlogits": d, "loss": loss}


def run(state):
    if own:
        return _own_run(state)
    return {"logprob": _plain_run_logprob, "logprob_grad": _plain_run_logprob_grad,
            "distill": _plain_run_distill, "distill_grad": _plain_run_distill_grad}[state["op"]](state)


# ------------------------------------------------------------------ 64 bits


def _exact_rows(st, x, part):
    """The outputs of the rows x [r, V] in float64; part picks the rows of a row input."""
    c, V = st["scale"], x.shape[-1]
    x = x.double()
    p = torch.softmax(x * c, -1)
    lse = torch.logsumexp(x * c, -1)
    if st["op"].startswith("logprob"):
        tok = part(st["tokens"]).long()
        ok = (tok != st["pad"]) & (tok >= 0) & (tok < V)
        hot = torch.nn.functional.one_hot(tok.clamp(0, V - 1), V)
        xt = torch.where(hot > 0, x, 0.0).sum(-1)
        logprob = torch.where(ok, xt * c - lse, 0.0)
        log_p = torch.log_softmax(x * c, -1)
        entropy = torch.special.entr(p).sum(-1)
        if st["op"] == "logprob":
            out = {"logprob": logprob, "entropy": entropy, "lse": lse}
            if st["k"]:
                ids = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :st["k"]]
                out["top_logprob"] = torch.take_along_dim(log_p, ids, -1)
                out["top_ids"] = ids.to(torch.int32)
            return out
        a = (part(st["g_logprob"]).double() * ok).unsqueeze(-1)
        b = part(st["g_entropy"]).double().unsqueeze(-1)
        surprise = torch.where(p > 0, log_p, 0.0) + entropy.unsqueeze(-1)
        return {"dlogits": c * (a * hot - a * p - b * p * surprise), "logprob": logprob,
                "entropy": entropy}
    ids, t = part(st["ids"]).long(), part(st["teacher"]).double()
    ok = ids >= 0
    has = ok.any(-1)
    t = torch.where(ok, t, -math.inf)
    if st["tail"]:
        q = t.exp()
        qr = (1.0 - q.sum(-1)).clamp_min(0.0) * has
    else:
        q = torch.softmax(torch.where(has.unsqueeze(-1), t, 0.0), -1) * ok
        qr = torch.zeros_like(lse)
    want = torch.zeros_like(x).scatter_add_(-1, ids.clamp_min(0), q)  # the teacher over V
    inside = torch.zeros_like(x).scatter_add_(-1, ids.clamp_min(0), ok.double()) > 0
    logp_at = torch.gather(x * c - lse.unsqueeze(-1), -1, ids.clamp_min(0))
    loss = torch.special.xlogy(q, q).sum(-1) - torch.where(q > 0, q * logp_at, 0.0).sum(-1)
    out = {}
    soft_rest = torch.zeros_like(x)
    if st["tail"]:
        outside = torch.where(inside, -math.inf, x * c)
        lse_rest = torch.logsumexp(outside, -1)
        soft_rest = torch.softmax(outside, -1)
        loss = loss + torch.where(qr > 0, torch.special.xlogy(qr, qr) - qr * (lse_rest - lse), 0.0)
    if st["op"] == "distill_grad":
        mass = (q.sum(-1) + qr).unsqueeze(-1)
        d = mass * p - want - qr.unsqueeze(-1) * soft_rest
        out["dlogits"] = d * (c * part(st["g"]).double()).unsqueeze(-1)
    out["loss"] = loss
    return out


def exact(case, seed):
    st = prepare(case, seed)
    x = st["logits"]
    lead = x.shape[:-1]
    per_step = x[0].numel()
    steps = max(1, (64 << 20) // max(1, per_step))
    parts = []
    for s0 in range(0, lead[0], steps):
        xs = x[s0:s0 + steps]

        def part(v, s0=s0):
            v = v[s0:s0 + steps]
            return v.reshape(-1, *v.shape[len(lead):])

        got = _exact_rows(st, xs.reshape(-1, x.shape[-1]), part)
        parts.append({key: v.reshape(*xs.shape[:-1], *v.shape[1:]) for key, v in got.items()})
    return {key: torch.cat([p[key] for p in parts]) for key in parts[0]}
