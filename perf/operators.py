"""Cases that measure the operators around the top-k in a decoding step: the gate that
chooses a token's experts, the verification of drafted tokens, and a cache in 4 bits with
the attention that reads it.

Each case names an operator ("op") and its sizes.  With ``own`` false ``run`` computes the
operator in elementary torch operations in fp32; with ``own`` true it calls the library."""
import math

import torch

own = False


# ------------------------------------------------------------------ the cases ----

def listed():
    return [
        # one decoding step's tokens at a gate of many experts in groups, sigmoid scores
        # and a balancing bias
        dict(name="route_decode", op="route", T=33, E=256, k=8, scoring="sigmoid", bias=True, groups=8, topk_groups=4,
             renorm=True, dtype="float32", train=False),
        # a training step's tokens at a gate with plain softmax weights, few experts, their
        # number no power of two
        dict(name="route_train_softmax", op="route", T=8190, E=60, k=4, scoring="softmax", bias=False, groups=1,
             topk_groups=1, renorm=False, dtype="bfloat16", train=True),
        # a training step's tokens at the large gate, with its backward pass and the load
        # of each expert
        dict(name="route_train_groups", op="route", T=16384, E=256, k=8, scoring="sigmoid", bias=True, groups=8,
             topk_groups=4, renorm=True, dtype="float32", train=True),
        # a single user's step with a draft model: latency
        dict(name="verify_one", op="verify", B=1, S=4, V=129280, dtype="float32", probs=True, agree=0.8, ragged=False),
        # a serving batch with a draft model, the sampler's vocabulary
        dict(name="verify_batch", op="verify", B=64, S=3, V=129280, dtype="float32", probs=True, agree=0.7, ragged=False),
        # a large batch whose drafts are looked up in the prompt (no draft probabilities),
        # bf16 logits, rows of an odd length, some requests with fewer drafts or none
        dict(name="verify_lookup", op="verify", B=200, S=5, V=32003, dtype="bfloat16", probs=False, agree=0.6, ragged=True),
        # a decoding batch's new keys and values
        dict(name="store_decode", op="store", T=64, H=8, D=128, page=64, dtype="bfloat16"),
        # a prompt's keys and values, and the same span read back
        dict(name="store_prompt", op="store", T=16411, H=8, D=128, page=64, dtype="bfloat16"),
        # a single user's step over a short context: latency
        dict(name="attend_one", op="attend", B=1, Q=1, Hq=32, H=8, D=128, L=4096, K=0, page=64, dtype="bfloat16",
             ragged=False),
        # a serving batch of four tokens (three drafts) a sequence, contexts of every length
        dict(name="attend_drafts", op="attend", B=48, Q=4, Hq=32, H=8, D=128, L=8192, K=0, page=64, dtype="bfloat16",
             ragged=True),
        # the indexer's shape: 512 selected positions out of 131072 for each of 64 rows
        dict(name="attend_selected", op="attend", B=64, Q=1, Hq=32, H=2, D=128, L=131072, K=512, page=64,
             dtype="bfloat16", ragged=False),
        # the long-context shape, read whole: one key and value head shared by 16 query heads
        dict(name="attend_long", op="attend", B=4, Q=1, Hq=16, H=1, D=128, L=1048576, K=0, page=128, dtype="bfloat16",
             ragged=False),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: an operator, then sizes over its whole range."""
    op = rng.choice(["route", "verify", "store", "attend", "attend"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
    if op == "route":  # one expert's renormalised weight is constant: nothing to learn from
        scoring = rng.choice(["softmax", "sigmoid"])
        groups = rng.choice([1, 1, 4, 8])
        size = rng.choice([8, 20, 32]) if groups > 1 else rng.choice([8, 60, 64, 72, 128, 160, 255, 256, 384, 512])
        k = rng.choice([1, 2, 4, 6, 8])
        return dict(op=op, T=_log_uniform(rng, 1, 16384), E=groups * size, k=k, scoring=scoring,
                    bias=scoring == "sigmoid" and rng.random() < 0.7, groups=groups,
                    topk_groups=1 if groups == 1 else rng.choice([1, groups // 2, groups - 1]),
                    renorm=k > 1 and rng.random() < 0.6, dtype=dtype, train=rng.random() < 0.5)
    if op == "verify":
        B, S = _log_uniform(rng, 1, 64), rng.randint(1, 6)
        V = min(_log_uniform(rng, 500, 160000), 35_000_000 // (B * (S + 1)))
        return dict(op=op, B=B, S=S, V=V, dtype=dtype, probs=rng.random() < 0.6, agree=rng.choice([0.3, 0.6, 0.9]),
                    ragged=rng.random() < 0.5)
    if op == "store":
        return dict(op=op, T=_log_uniform(rng, 1, 16384), H=rng.choice([1, 2, 8]), D=rng.choice([64, 128]),
                    page=rng.choice([16, 64, 128]), dtype=dtype)
    H = rng.choice([1, 2, 4, 8])
    B, Q = _log_uniform(rng, 1, 48), rng.choice([1, 1, 2, 5])
    L = min(_log_uniform(rng, 1, 131072), 2_000_000 // (B * H))
    return dict(op=op, B=B, Q=Q, Hq=H * rng.choice([1, 4, 8, 16]), H=H, D=rng.choice([64, 128]), L=max(L, Q),
                K=rng.choice([0, 0, _log_uniform(rng, 16, 2048)]), page=rng.choice([16, 64, 128]), dtype=dtype,
                ragged=rng.random() < 0.7)


def _es(case):
    return 4 if case["dtype"] == "float32" else 2


def work(case):
    op, es = case["op"], _es(case)
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        b, f = T * E * es + T * k * 8 + (4 * E if case["bias"] else 0), 4 * T * E
        if case["train"]:  # the gradient's output, the weights' gradient, the load of each expert
            b, f = b + T * E * es + T * k * 4 + 4 * E, f + 2 * T * E
        return {"bytes": b, "flops": f}
    if op == "verify":
        # rows after the first refused draft have no part in the answer: the expected number
        # of rows up to it, one row of the noise, and one of the draft's probabilities where
        # a draft was refused
        B, S, V, a = case["B"], case["S"], case["V"], case["agree"]
        drafts = [n for n in range(S + 1)] if case["ragged"] else [S]
        rows = B * sum((1 - a ** (n + 1)) / (1 - a) for n in drafts) / len(drafts)
        refused = B * sum(1 - a ** n for n in drafts) / len(drafts)
        return {"bytes": int(rows * V * es + B * V * 4 + (refused * V * 4 if case["probs"] else 0)),
                "flops": int(6 * rows * V)}
    if op == "store":
        T, H, D = case["T"], case["H"], case["D"]
        return {"bytes": 2 * (T * H * 2 * D * es + T * H * (D + 8)), "flops": 8 * T * H * D}
    B, Q, Hq, H, D, L, K = (case[n] for n in ("B", "Q", "Hq", "H", "D", "L", "K"))
    mean = (L + 1) // 2 if case["ragged"] else L
    seen = B * Q * min(K, mean) if K else B * mean  # cache entries read
    per = B * Q * (min(K, mean) if K else mean)     # positions each query token attends to
    return {"bytes": seen * H * (D + 8) + B * Q * Hq * (2 * D * es + 4) + 4 * B * Q * K, "flops": 4 * per * Hq * D}


# ------------------------------------------------------------------ inputs -------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _quantise(x):
    """Codes 0..15 (uint8, one each) and (scale, minimum) in bf16 of each row of x (fp32)."""
    m = x.amin(-1, keepdim=True).bfloat16().float()
    s = ((x.amax(-1, keepdim=True) - m) * (1.0 / 15.0)).bfloat16().float()
    inv = torch.where(s >= 2.0 ** -126, torch.ones_like(s) / s, torch.zeros_like(s))
    codes = torch.round((x - m) * inv).clamp(0, 15).to(torch.uint8)
    return codes, torch.cat([s, m], -1).bfloat16()


def _pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _unpack(packed):
    return torch.stack([packed & 15, packed >> 4], -1).flatten(-2)


def prepare(case, seed):
    g = _gen(seed)
    dt = getattr(torch, case["dtype"])
    st = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        st["logits"] = (1.5 * normal(T, E)).to(dt)
        st["bias"] = 0.05 * normal(E) if case["bias"] else None
        st["grad"] = normal(T, k) if case["train"] else None
        st["counts"] = case["train"]
    elif case["op"] == "verify":
        # the target: normal logits with a few likely tokens a row; the draft agrees with it
        # with the case's probability (its distribution is the target's mixed with another)
        B, S, V = case["B"], case["S"], case["V"]

        def logits():
            x = 2.0 * normal(B, S + 1, V)
            at = torch.randint(V, (B, S + 1, 4), device="cuda", generator=g)
            top = 8.0 + 4.0 * torch.rand(B, S + 1, 4, device="cuda", generator=g) + math.log(V / 1e4)
            return x.scatter_(2, at, top)
        x = logits().to(dt)
        st["logits"] = x
        temp = 0.5 + torch.rand(B, device="cuda", generator=g)
        if B >= 8:
            temp[3] = 0.0  # a request that asks for the likeliest token
        st["temperature"] = temp
        p = torch.softmax(x[:, :S].float() / temp.clamp(min=0.05)[:, None, None], -1)
        if case["probs"]:
            other = torch.softmax(logits()[:, :S], -1)
            q = case["agree"] * p + (1 - case["agree"]) * other
            st["q"] = q
            race = torch.empty_like(q).exponential_(generator=g)
            st["drafts"] = (q / race).argmax(-1).int()
            del other, race
        else:
            # a looked-up token: the likeliest one as often as drafts agree
            guess = torch.randint(V, (B, S), device="cuda", generator=g)
            hit = torch.rand(B, S, device="cuda", generator=g) < case["agree"]
            st["q"] = None
            st["drafts"] = torch.where(hit, p.argmax(-1), guess).int()
        st["lens"] = torch.randint(S + 1, (B,), device="cuda", generator=g).int() if case["ragged"] else None
        st["uniforms"] = torch.rand(B, S, device="cuda", generator=g)
        st["noise"] = torch.empty(B, V, device="cuda").exponential_(generator=g).clamp_(min=1e-10)
    elif case["op"] == "store":
        T, H, D, page = (case[n] for n in ("T", "H", "D", "page"))
        pages = -(-T // page) + 3
        st["k"], st["v"] = normal(T, H, D).to(dt), normal(T, H, D).to(dt)
        st["cache"] = torch.zeros(pages, H, page, 2, D // 2, dtype=torch.uint8, device="cuda")
        st["scales"] = torch.zeros(pages, H, page, 4, dtype=torch.bfloat16, device="cuda")
        # pages in any order, a first page that is partly filled already
        order = torch.randperm(pages, device="cuda", generator=g)
        at = torch.arange(T, device="cuda") + page // 3
        st["slots"] = (order[at // page] * page + at % page).int()
    else:
        B, Q, Hq, H, D, L, K, page = (case[n] for n in ("B", "Q", "Hq", "H", "D", "L", "K", "page"))
        per = -(-L // page)
        pages = B * per
        st["q"] = (1.5 * normal(B, Q, Hq, D)).to(dt)
        st["cache"] = torch.empty(pages, H, page, 2, D // 2, dtype=torch.uint8, device="cuda")
        st["scales"] = torch.empty(pages, H, page, 4, dtype=torch.bfloat16, device="cuda")
        step = max(1, (1 << 27) // (H * page * 2 * D))
        for i in range(0, pages, step):
            codes, sc = _quantise(normal(min(step, pages - i), H, page, 2, D))
            st["cache"][i:i + step] = _pack(codes)
            st["scales"][i:i + step] = sc.flatten(-2)
        st["table"] = torch.randperm(pages, device="cuda", generator=g).view(B, per).int()
        lens = torch.full((B,), L, device="cuda")
        if case["ragged"]:
            lens = torch.randint(L + 1, (B,), device="cuda", generator=g)
        st["lens"] = lens.int()
        st["indices"] = None
        if K:  # distinct positions in no order, -1 behind the last where the context is shorter
            score = torch.rand(B, Q, L, device="cuda", generator=g)
            ends = lens[:, None] - (Q - 1) + torch.arange(Q, device="cuda")
            score.masked_fill_(torch.arange(L, device="cuda") >= ends[..., None], -1.0)
            top, idx = score.topk(min(K, L), -1)
            idx = torch.where(top >= 0, idx, -1)
            if K > L:
                idx = torch.cat([idx, torch.full((B, Q, K - L), -1, device="cuda")], -1)
            st["indices"] = idx.int().contiguous()
    return st


# ------------------------------------------------------------------ plain forms --

def _first_max(x):
    """The lowest index of each row's largest value."""
    at = torch.arange(x.shape[-1], device=x.device)
    return torch.where(x == x.amax(-1, keepdim=True), at, x.shape[-1]).amin(-1)


def _plain_route(st):
    c = st["case"]
    x = st["logits"].float()
    if c["scoring"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(-1, keepdim=True))
        s = e / e.sum(-1, keepdim=True)
    # the scores rise with the logits: without a bias the choice goes by the logits
    choice = x if st["bias"] is None else s + st["bias"]
    if c["groups"] > 1:
        T, E = x.shape
        by = choice.view(T, c["groups"], -1)
        if st["bias"] is None:
            score = by.amax(-1)
        else:
            top = by.sort(dim=-1, descending=True, stable=True).values
            score = top[..., 0] + top[..., 1]
        best = score.sort(dim=-1, descending=True, stable=True).indices[:, :c["topk_groups"]]
        keep = torch.zeros_like(score, dtype=torch.bool).scatter_(1, best, True)
        choice = by.masked_fill(~keep[..., None], -math.inf).view(T, E)
    experts = choice.sort(dim=-1, descending=True, stable=True).indices[:, :c["k"]]
    chosen = s.gather(1, experts)
    total = chosen.sum(-1, keepdim=True) if c["renorm"] else torch.ones_like(chosen[:, :1])
    out = {"weights": 2.5 * chosen / total, "experts": experts.int()}
    if c["train"]:
        out["counts"] = torch.zeros(c["E"], dtype=torch.int32, device="cuda").index_add_(
            0, experts.flatten(), torch.ones(experts.numel(), dtype=torch.int32, device="cuda"))
        g = st["grad"]
        mean = (g * chosen / total).sum(-1, keepdim=True) if c["renorm"] else 0.0
        ds = 2.5 * (g - mean) / total
        full = torch.zeros_like(x).scatter_(1, experts, ds)
        if c["scoring"] == "sigmoid":
            dx = full * s * (1.0 - s)
        else:
            dx = s * (full - (full * s).sum(-1, keepdim=True))
        out["grad_logits"] = dx.to(st["logits"].dtype)
    return out


def _plain_verify(st):
    x = st["logits"].float()
    B, rows, V = x.shape
    S = rows - 1
    t = st["temperature"][:, None, None]
    greedy = t <= 0
    e = torch.exp((x - x.amax(-1, keepdim=True)) / torch.where(greedy, torch.ones_like(t), t))
    p = e / e.sum(-1, keepdim=True)
    hot = torch.zeros_like(p).scatter_(2, _first_max(x)[..., None], 1.0)
    p = torch.where(greedy, hot, p)
    drafts = st["drafts"].long()
    lens = torch.full((B,), S, device="cuda") if st["lens"] is None else st["lens"].long()
    p_at = p[:, :S].gather(2, drafts[..., None])[..., 0]
    q_at = torch.ones_like(p_at) if st["q"] is None else st["q"].gather(2, drafts[..., None])[..., 0]
    ok = (st["uniforms"] * q_at < p_at) & (torch.arange(S, device="cuda") < lens[:, None])
    n = ok.int().cumprod(-1).sum(-1)
    at = torch.arange(B, device="cuda")
    stop = p[at, n]
    refused = n.clamp(max=S - 1)
    if st["q"] is None:
        q = torch.zeros_like(stop).scatter_(1, drafts[at, refused][:, None], 1.0)
    else:
        q = st["q"][at, refused]
    rest = torch.where((n < lens)[:, None], (stop - q).clamp(min=0.0), stop)
    rest = torch.where(rest.amax(-1, keepdim=True) > 0, rest, stop)
    last = _first_max(rest / st["noise"])
    place = torch.arange(rows, device="cuda")
    padded = torch.cat([drafts, torch.zeros_like(drafts[:, :1])], 1)
    probs = torch.cat([p_at, torch.zeros_like(p_at[:, :1])], 1)
    tokens = torch.where(place < n[:, None], padded, torch.where(place == n[:, None], last[:, None], -1))
    probs = torch.where(place < n[:, None], probs, torch.where(place == n[:, None], stop.gather(1, last[:, None]), 0.0))
    return {"tokens": tokens.int(), "accepted": n.int(), "probs": probs}


def _plain_store(st):
    page = st["cache"].shape[2]
    slots = st["slots"].long()
    codes, sc = _quantise(torch.stack([st["k"].float(), st["v"].float()], 2))
    st["cache"][slots // page, :, slots % page] = _pack(codes)
    st["scales"][slots // page, :, slots % page] = sc.flatten(-2)
    back = _unpack(st["cache"][slots // page, :, slots % page]).float()
    sc = st["scales"][slots // page, :, slots % page].float().unflatten(-1, (2, 2))
    back = (back * sc[..., :1] + sc[..., 1:]).to(st["k"].dtype)
    return {"k": back[:, :, 0], "v": back[:, :, 1]}


def _plain_attend(st):
    c = st["case"]
    q = st["q"].float()
    B, Q, Hq, D = q.shape
    H, page = st["cache"].shape[1:3]
    G = Hq // H
    lens, table = st["lens"].long(), st["table"].long()
    ends = lens[:, None] - (Q - 1) + torch.arange(Q, device="cuda")  # [B, Q]: positions each token sees
    if st["indices"] is None:
        def whole(t):  # [B, H, positions, ...] of pages [pages, H, page, ...]
            return t[table].transpose(1, 2).flatten(2, 3)
        codes, sc = _unpack(whole(st["cache"])).float(), whole(st["scales"]).float()
        there = torch.arange(codes.shape[2], device="cuda") < ends[..., None]
        there = there[:, None, :, None].expand(B, H, Q, G, -1).reshape(B, H, Q * G, -1)
        x = q.view(B, Q, H, G, D).transpose(1, 2).reshape(B, H, Q * G, D)
    else:
        idx = st["indices"].long()
        there = (idx >= 0) & (idx < ends[..., None])
        pos = torch.where(there, idx, 0)
        pg = table[torch.arange(B, device="cuda")[:, None, None], pos // page]

        def picked(t):  # [B, Q, H, K, ...]
            return t[pg, :, pos % page].transpose(2, 3)
        codes, sc = _unpack(picked(st["cache"])).float(), picked(st["scales"]).float()
        there = there[:, :, None, None]
        x = q.view(B, Q, H, G, D)
    sc = sc.unflatten(-1, (2, 2))
    kv = codes * sc[..., :1] + sc[..., 1:]
    s = (x * (1.0 / math.sqrt(D))) @ kv[..., 0, :].transpose(-1, -2)
    s = s.masked_fill(~there, -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(s - m)
    l = p.sum(-1, keepdim=True)
    out = (p @ kv[..., 1, :]) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + torch.log(l))[..., 0]
    if st["indices"] is None:
        out = out.view(B, H, Q, G, D).transpose(1, 2)
        lse = lse.view(B, H, Q, G).transpose(1, 2)
    return {"out": out.reshape(B, Q, Hq, D).to(st["q"].dtype), "lse": lse.reshape(B, Q, Hq)}


def run(st):
    c = st["case"]
    if not own:
        return {"route": _plain_route, "verify": _plain_verify, "store": _plain_store, "attend": _plain_attend}[c["op"]](st)
    import top_selection_gb300 as ds
    if c["op"] == "route":
        counts = torch.zeros(c["E"], dtype=torch.int32, device="cuda") if c["train"] else None
        w, e = ds.route(st["logits"], c["k"], scoring=c["scoring"], bias=st["bias"], groups=c["groups"],
                        topk_groups=c["topk_groups"], group_score="max" if st["bias"] is None else "top2",
                        renormalise=c["renorm"], scale=2.5, counts=counts)
        out = {"weights": w, "experts": e}
        if c["train"]:
            out["counts"] = counts
            out["grad_logits"] = ds.route_backward(st["grad"], st["logits"], e, scoring=c["scoring"],
                                                   renormalise=c["renorm"], scale=2.5)
        return out
    if c["op"] == "verify":
        tokens, accepted, probs = ds.verify_drafts(st["logits"], st["drafts"], st["uniforms"], st["noise"],
                                                   draft_probs=st["q"], draft_lens=st["lens"],
                                                   temperature=st["temperature"])
        return {"tokens": tokens, "accepted": accepted, "probs": probs}
    if c["op"] == "store":
        ds.cache_store(st["k"], st["v"], st["cache"], st["scales"], st["slots"])
        k, v = ds.cache_load(st["cache"], st["scales"], st["slots"], dtype=st["k"].dtype)
        return {"k": k, "v": v}
    out, lse = ds.cache_attention(st["q"], st["cache"], st["scales"], st["table"], st["lens"], indices=st["indices"])
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ in 64 bits ---

def _exact_route(c, st):
    x = st["logits"].double()
    b = None if st["bias"] is None else st["bias"].double()
    s = torch.sigmoid(x) if c["scoring"] == "sigmoid" else torch.softmax(x, -1)
    key = x.clone() if b is None else s + b
    T, E = x.shape
    if c["groups"] > 1:
        size = E // c["groups"]
        scores = []
        for i in range(c["groups"]):
            part = key[:, i * size:(i + 1) * size]
            scores.append(part.topk(1 if b is None else 2, -1).values.sum(-1))
        order = torch.stack(scores, 1).argsort(dim=-1, descending=True, stable=True)
        for j in range(c["topk_groups"], c["groups"]):
            lost = order[:, j:j + 1] * size + torch.arange(size, device="cuda")
            key.scatter_(1, lost, -math.inf)
    experts = key.argsort(dim=-1, descending=True, stable=True)[:, :c["k"]]
    w = s.gather(1, experts)
    norm = w.sum(-1, keepdim=True) if c["renorm"] else torch.ones(T, 1, dtype=x.dtype, device="cuda")
    out = {"weights": 2.5 * w / norm, "experts": None}
    if c["train"]:
        g = st["grad"].double()
        if c["renorm"]:  # dw_i/ds_j = scale (delta_ij - w_i / norm) / norm
            ds = 2.5 * (g / norm - (g * w).sum(-1, keepdim=True) / norm ** 2)
        else:
            ds = 2.5 * g
        if c["scoring"] == "sigmoid":
            dx = torch.zeros_like(x).scatter_(1, experts, ds * w * (1 - w))
        else:  # ds_i/dx_e = s_i (delta_ie - s_e)
            dx = -s * (ds * w).sum(-1, keepdim=True)
            dx.scatter_add_(1, experts, ds * w)
        out["counts"], out["grad_logits"] = None, dx
    return out


def _exact_verify(c, st):
    B, S = c["B"], c["S"]
    probs = torch.zeros(B, S + 1, dtype=torch.float64, device="cuda")
    for b in range(B):
        t = float(st["temperature"][b])
        limit = S if st["lens"] is None else int(st["lens"][b])
        for i in range(S + 1):
            x = st["logits"][b, i].double()
            if t > 0:
                p = torch.softmax(x / t, -1)
            else:
                p = torch.zeros_like(x)
                p[int((x == x.max()).nonzero()[0])] = 1.0
            if i < limit:
                d = int(st["drafts"][b, i])
                q = None if st["q"] is None else st["q"][b, i].double()
                if float(st["uniforms"][b, i]) * (1.0 if q is None else float(q[d])) < float(p[d]):
                    probs[b, i] = p[d]
                    continue
                if q is None:
                    q = torch.zeros_like(p)
                    q[d] = 1.0
                r = (p - q).clamp(min=0)
                r = r if float(r.max()) > 0 else p
            else:
                r = p
            probs[b, i] = p[int((r / st["noise"][b].double()).argmax())]
            break
    return {"tokens": None, "accepted": None, "probs": probs}


def _exact_store(c, st):
    out = {}
    for name in ("k", "v"):
        x = st[name].double()
        m = x.min(-1, keepdim=True).values.to(torch.bfloat16).double()
        s = ((x.max(-1, keepdim=True).values - m) / 15).to(torch.bfloat16).double()
        out[name] = m + s * torch.round((x - m) / s).clamp(0, 15)
    return out


def _exact_attend(c, st):
    B, Q, Hq, H, D = (c[n] for n in ("B", "Q", "Hq", "H", "D"))
    page, G = c["page"], Hq // H
    out = torch.zeros(B, Q, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((B, Q, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for b in range(B):
        n = int(st["lens"][b])
        for i in range(Q):
            end = n - (Q - 1 - i)
            if st["indices"] is None:
                pos = torch.arange(max(end, 0), device="cuda")
            else:
                pos = st["indices"][b, i].long()
                pos = pos[(pos >= 0) & (pos < end)]
            if pos.numel() == 0:
                continue
            pg, off = st["table"][b].long()[pos // page], pos % page
            for h in range(H):
                raw, sc = st["cache"][pg, h, off], st["scales"][pg, h, off].double()
                low, high = (raw & 15).double(), (raw >> 4).double()
                code = torch.empty(*raw.shape[:-1], D, dtype=torch.float64, device="cuda")
                code[..., 0::2], code[..., 1::2] = low, high
                k = code[:, 0] * sc[:, 0:1] + sc[:, 1:2]
                v = code[:, 1] * sc[:, 2:3] + sc[:, 3:4]
                s = st["q"][b, i, h * G:(h + 1) * G].double() @ k.T / math.sqrt(D)
                z = torch.logsumexp(s, -1)
                lse[b, i, h * G:(h + 1) * G] = z
                out[b, i, h * G:(h + 1) * G] = torch.exp(s - z[:, None]) @ v
    return {"out": out, "lse": lse}


def exact(case, seed):
    st = prepare(case, seed)
    return {"route": _exact_route, "verify": _exact_verify, "store": _exact_store, "attend": _exact_attend}[case["op"]](case, st)
