"""Cases that measure what follows the selections: the log probabilities of given tokens with
entropy and likeliest alternatives, the exchange that sorts tokens by their chosen experts and
brings the experts' outputs back, the 8-bit form of rows and weights with a scale for each block
of 128, and the experts' products in that form.

Each case names an operator ("op") and its sizes.  With ``own`` false ``run`` computes the
operator in elementary torch operations in fp32; with ``own`` true it calls the library."""
import math

import torch

own = False


# ------------------------------------------------------------------ the cases ----

def listed():
    return [
        # one row of a decoding step's logits, with the 20 likeliest tokens beside the drawn
        # one: latency
        dict(name="logprobs_one", op="logprobs", T=1, V=129280, top=20, dtype="float32", train=False),
        # a serving batch that asks for its tokens' log probabilities and five alternatives
        dict(name="logprobs_batch", op="logprobs", T=256, V=129280, top=5, dtype="float32", train=False),
        # a prompt scored whole: bf16 rows of an odd length, the likeliest token beside each
        dict(name="logprobs_prompt", op="logprobs", T=4099, V=32003, top=1, dtype="bfloat16", train=False),
        # a step of training on drawn tokens: log probabilities and entropies, and the gradient
        # of both, some tokens left out
        dict(name="logprobs_train", op="logprobs", T=2048, V=129280, top=0, dtype="bfloat16", train=True),
        # one decoding step's tokens sorted for the experts in 8 bits, and the outputs back
        dict(name="exchange_decode", op="exchange", T=33, E=256, k=8, D=2048, dtype="bfloat16", padded=False,
             quantise=True, train=False),
        # a padded batch in fp32, few experts, rows of an odd length, with gradients
        dict(name="exchange_padded", op="exchange", T=4093, E=60, k=4, D=1001, dtype="float32", padded=True,
             quantise=False, train=True),
        # a training step's tokens at the large gate, forth and back, with all gradients
        dict(name="exchange_train", op="exchange", T=16384, E=256, k=8, D=2048, dtype="bfloat16", padded=False,
             quantise=False, train=True),
        # a prompt's activations to 8 bits, a scale for each 128 numbers of a row
        dict(name="quantise_rows", op="quantise", E=1, N=16411, K=2048, block=1, dtype="bfloat16"),
        # the experts' weights to 8 bits, a scale for each block of 128 x 128
        dict(name="quantise_weights", op="quantise", E=16, N=2000, K=4096, block=128, dtype="float32"),
        # one token through a dense layer in 8 bits: latency and the weights' bytes
        dict(name="product_one", op="product", T=1, E=1, N=4096, K=4096, skew=0.0, dtype="bfloat16"),
        # a decoding batch's choices (64 tokens, 8 experts each) over 64 experts of unlike load
        dict(name="product_decode", op="product", T=512, E=64, N=2048, K=4096, skew=1.0, dtype="bfloat16"),
        # a prompt's choices over 64 experts, the products' operations
        dict(name="product_prompt", op="product", T=32768, E=64, N=4096, K=2048, skew=0.5, dtype="bfloat16"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: an operator, then sizes over its whole range."""
    op = rng.choice(["logprobs", "exchange", "quantise", "product", "product"])
    dtype = rng.choice(["bfloat16", "bfloat16", "float32"])
    if op == "logprobs":
        T = _log_uniform(rng, 1, 4096)
        V = min(_log_uniform(rng, 100, 200000), 130_000_000 // T)
        train = rng.random() < 0.4
        return dict(op=op, T=T, V=V, top=0 if train else min(V, rng.choice([0, 1, 5, 20, 32])), dtype=dtype, train=train)
    if op == "exchange":
        E = rng.choice([4, 8, 60, 64, 128, 160, 256, 512])
        k = rng.choice([1, 2, 4, 6, 8])
        T = _log_uniform(rng, 1, 16384)
        D = min(_log_uniform(rng, 64, 6000), 400_000_000 // (T * k * (4 if dtype == "float32" else 2)))
        train = rng.random() < 0.5
        return dict(op=op, T=T, E=E, k=min(k, E), D=D, dtype=dtype, padded=rng.random() < 0.4,
                    quantise=not train and rng.random() < 0.5, train=train)
    if op == "quantise":
        E, block = rng.choice([1, 1, 3, 16]), rng.choice([1, 128])
        N, K = _log_uniform(rng, 1, 8192), _log_uniform(rng, 16, 8192)
        return dict(op=op, E=E, N=min(N, max(1, 130_000_000 // (E * K))), K=K, block=block, dtype=dtype)
    E = rng.choice([1, 1, 8, 32, 64, 160])
    K, N = 16 * _log_uniform(rng, 4, 512), _log_uniform(rng, 32, 6000)
    N = min(N, 400_000_000 // (E * K))
    T = min(_log_uniform(rng, 1, 16384), 270_000_000_000 // (N * K))
    return dict(op=op, T=T, E=E, N=N, K=K, skew=rng.choice([0.0, 0.5, 2.0]), dtype=dtype)


def _es(case):
    return 4 if case["dtype"] == "float32" else 2


def work(case):
    op, es = case["op"], _es(case)
    if op == "logprobs":
        T, V = case["T"], case["V"]
        b, f = T * V * es + T * (16 + 8 * case["top"]), 6 * T * V
        if case["train"]:  # the logits once more and their gradient
            b, f = b + 2 * T * V * es + 24 * T, f + 6 * T * V
        return {"bytes": b, "flops": f}
    if op == "exchange":
        T, k, D, E = (case[n] for n in ("T", "k", "D", "E"))
        n = T * k
        # experts, places, offsets; tokens read, their sorted rows written, the experts' outputs
        # and weights read, the tokens' sums written
        out = D + 4 * ((D + 127) // 128) if case["quantise"] else D * es
        b, f = 8 * n + 4 * E + T * D * es + n * out + n * (D * es + 4) + T * D * es, 2 * n * D
        if case["train"]:
            # back through the sums: their gradient and the experts' outputs read, two
            # gradients written; back through the sorting: rows' gradients read, tokens' written
            b, f = b + 2 * T * D * es + 3 * n * D * es + 8 * n, f + 4 * n * D
        return {"bytes": b, "flops": f}
    if op == "quantise":
        E, N, K, c = case["E"], case["N"], case["K"], case["block"]
        return {"bytes": E * N * K * (es + 1) + 4 * E * -(-N // c) * -(-K // 128), "flops": 3 * E * N * K}
    T, E, N, K = (case[n] for n in ("T", "E", "N", "K"))
    # the weights of experts that have a row (the expected number of them where rows are few
    # and spread evenly), the rows, both scales, the products
    used = E * (1 - (1 - 1 / E) ** T) if E > 1 else 1
    kb = -(-K // 128)
    return {"bytes": int(used * (N * K + 4 * -(-N // 128) * kb)) + T * K + 4 * T * kb + T * N * es, "flops": 2 * T * N * K}


# ------------------------------------------------------------------ inputs -------

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _blocks(x, rows):
    """x (E, N, K) in whole blocks of rows x 128, zeros behind the edges: (E, n, rows, k, 128)."""
    E, N, K = x.shape
    n, k = -(-N // rows), -(-K // 128)
    return torch.nn.functional.pad(x, (0, 128 * k - K, 0, rows * n - N)).view(E, n, rows, k, 128)


def _spread(scales, rows, N, K):
    """A scale for each number: scales (E, n, k) over (E, N, K)."""
    return scales.repeat_interleave(rows, 1)[:, :N].repeat_interleave(128, 2)[:, :, :K]


def prepare(case, seed):
    g = _gen(seed)
    dt = getattr(torch, case["dtype"])
    st = {"case": case}

    def normal(*shape):
        return torch.randn(*shape, device="cuda", generator=g)

    if case["op"] == "logprobs":
        # normal logits with a few likely tokens a row; the given token is one of those three
        # times of four, any one otherwise
        T, V = case["T"], case["V"]
        x = torch.empty(T, V, device="cuda", dtype=dt)
        step = max(1, (1 << 26) // V)
        for i in range(0, T, step):
            x[i:i + step] = 2.0 * normal(min(step, T - i), V)
        at = torch.randint(V, (T, 4), device="cuda", generator=g)
        x.scatter_(1, at, (8.0 + 4.0 * torch.rand(T, 4, device="cuda", generator=g) + math.log(V / 1e4)).to(dt))
        any_one = torch.randint(V, (T,), device="cuda", generator=g)
        tokens = torch.where(torch.rand(T, device="cuda", generator=g) < 0.75, at[:, 0], any_one).int()
        if case["train"]:  # places that are not trained on: prompts, padding
            tokens = torch.where(torch.rand(T, device="cuda", generator=g) < 0.1, -1, tokens)
        st["logits"], st["tokens"] = x, tokens
        st["grad"] = normal(T) if case["train"] else None
        st["grad_entropy"] = 0.01 * normal(T) if case["train"] else None
    elif case["op"] == "exchange":
        T, E, k, D = (case[n] for n in ("T", "E", "k", "D"))
        # the choice of a gate whose experts are of unlike popularity
        score = normal(T, E) + 0.7 * normal(E)
        top, experts = score.topk(k, -1)
        experts = experts.int()
        if case["padded"]:  # the last rows of a batch, and a few within it
            off = torch.rand(T, device="cuda", generator=g) < 0.05
            off[T - T // 8:] = True
            experts[off] = -1
        st["experts"], st["weights"] = experts, torch.softmax(top, -1).contiguous()
        st["x"] = normal(T, D).to(dt)
        st["y"] = torch.empty(T * k, D, device="cuda", dtype=dt).normal_(generator=g)
        st["grad"] = normal(T, D).to(dt) if case["train"] else None
        st["grad_rows"] = torch.empty(T * k, D, device="cuda", dtype=dt).normal_(generator=g) if case["train"] else None
    elif case["op"] == "quantise":
        E, N, K = case["E"], case["N"], case["K"]
        # rows of unlike size, a few large numbers among them
        x = torch.empty(E, N, K, device="cuda").normal_(generator=g) * torch.exp(normal(E, N, 1))
        x.view(-1)[torch.randint(x.numel(), (max(1, x.numel() // 1000),), device="cuda", generator=g)] *= 20.0
        st["x"] = x.to(dt)
    else:
        T, E, N, K, skew = (case[n] for n in ("T", "E", "N", "K", "skew"))
        # rows as the quantiser gives them (powers of two for scales), weights as a checkpoint
        # holds them (any scales)
        x = normal(1, T, K)
        top = _blocks(x, 1).abs().amax((2, 4))
        sx = torch.exp2(torch.ceil(torch.log2(top.clamp(min=1e-30) / 448.0)))
        st["x"], st["x_scales"] = (x / _spread(sx, 1, T, K))[0].to(torch.float8_e4m3fn), sx[0].contiguous()
        w = torch.empty(E, N, K, device="cuda", dtype=torch.float8_e4m3fn)
        sw = torch.empty(E, -(-N // 128), -(-K // 128), device="cuda")
        for e in range(E):
            v = normal(1, N, K) * K ** -0.5
            s = _blocks(v, 128).abs().amax((2, 4)) / 448.0
            w[e], sw[e] = (v / _spread(s, 128, N, K))[0].to(torch.float8_e4m3fn), s[0]
        st["w"], st["w_scales"] = w, sw
        # how many rows each expert has: shares that differ by exp(skew) of a standard deviation
        share = torch.softmax(skew * normal(E), -1)
        counts = torch.bincount(torch.multinomial(share, T, replacement=True, generator=g), minlength=E)
        offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
        offsets[1:] = counts.cumsum(0)
        st["offsets"], st["ends"] = offsets.int(), offsets.tolist()
    return st


# ------------------------------------------------------------------ plain forms --

def _plain_logprobs(st):
    c = st["case"]
    x = st["logits"].float()
    T, V = x.shape
    m = x.amax(-1, keepdim=True)
    y = x - m
    e = torch.exp(y)
    s = e.sum(-1, keepdim=True)
    logs = torch.log(s)
    p = e / s
    tokens = st["tokens"].long()
    there = (tokens >= 0) & (tokens < V)
    at = torch.where(there, tokens, 0)[:, None]
    logp = y - logs
    logprob = torch.where(there, logp.gather(1, at)[:, 0], 0.0)
    entropy = logs[:, 0] - (p * y).sum(-1)
    out = {"logprobs": logprob, "lse": (m + logs)[:, 0], "entropy": entropy}
    if c["top"]:
        order = st["logits"].sort(dim=-1, descending=True, stable=True).indices[:, :c["top"]]
        out["top_logprobs"], out["top_tokens"] = logp.gather(1, order), order.int()
    if c["train"]:
        g = torch.where(there, st["grad"], 0.0)[:, None]
        # d logprob / dx = [given] - p;  d entropy / dx = -p (log p + entropy)
        dx = -p * (g + st["grad_entropy"][:, None] * (logp + entropy[:, None]))
        dx.scatter_add_(1, at, g)
        out["grad_logits"] = dx.to(st["logits"].dtype)
    return out


def _quantise(x, rows):
    """(codes, scales) of x (E, N, K) in fp32: the scale of a block is the least power of two (no
    less than 2^-126) that brings its largest number to 448 or below."""
    E, N, K = x.shape
    top = _blocks(x, rows).abs().amax((2, 4))
    part, power = torch.frexp(top)  # top = part * 2^power, part in [1/2, 1); 448 = 7/8 * 2^9
    power = power - 9 + (part > 0.875).int()
    power = torch.where(top > 0, power, -126).clamp(min=-126)
    scales = ((power + 127) << 23).view(torch.float32)
    return (x / _spread(scales, rows, N, K)).to(torch.float8_e4m3fn), scales


def _plain_exchange(st):
    c = st["case"]
    T, E, k, D = (c[n] for n in ("T", "E", "k", "D"))
    dt = st["x"].dtype
    experts = st["experts"].flatten().long()
    there = experts >= 0
    key = torch.where(there, experts, E)
    order = key.sort(stable=True).indices
    places = torch.empty_like(order)
    places[order] = torch.arange(T * k, device="cuda")
    counts = torch.zeros(E + 1, dtype=torch.int64, device="cuda").index_add_(0, key, torch.ones_like(key))
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = counts[:E].cumsum(0)
    full = (torch.arange(T * k, device="cuda") < offsets[E])[:, None]
    out = {"places": torch.where(there, places, -1).view(T, k).int(), "offsets": offsets.int()}
    x = torch.where(full, st["x"][order // k], 0.0)
    if c["quantise"]:
        codes, scales = _quantise(x.float()[None], 1)
        out["codes"], out["scales"] = codes[0], scales[0]
    else:
        out["rows"] = x.to(dt)
    there = there.view(T, k, 1)
    places = places.view(T, k)
    w = st["weights"][..., None]
    back = torch.where(there, st["y"][places].float(), 0.0)
    out["out"] = (w * back).sum(1).to(dt)
    if c["train"]:
        g = st["grad"].float()[:, None]
        out["grad_x"] = torch.where(there, st["grad_rows"][places].float(), 0.0).sum(1).to(dt)
        out["grad_weights"] = (g * back).sum(-1)
        grad_y = (w * g).view(T * k, D)[order]
        out["grad_y"] = torch.where(full, grad_y, 0.0).to(dt)
    return out


def _plain_quantise(st):
    codes, scales = _quantise(st["x"].float(), st["case"]["block"])
    return {"codes": codes, "scales": scales}


def _plain_product(st):
    c = st["case"]
    x = st["x"].float() * _spread(st["x_scales"][None], 1, c["T"], c["K"])[0]
    w = st["w"].float() * _spread(st["w_scales"], 128, c["N"], c["K"])
    ends = st["ends"]
    out = torch.cat([x[a:b] @ m.T for a, b, m in zip(ends[:-1], ends[1:], w)])
    return {"out": out.to(getattr(torch, c["dtype"]))}


def run(st):
    c = st["case"]
    if not own:
        return {"logprobs": _plain_logprobs, "exchange": _plain_exchange, "quantise": _plain_quantise,
                "product": _plain_product}[c["op"]](st)
    import top_selection_gb300 as ds
    if c["op"] == "logprobs":
        logprobs, lse, entropy, top_logprobs, top_tokens = ds.token_logprobs(st["logits"], st["tokens"], top=c["top"])
        out = {"logprobs": logprobs, "lse": lse, "entropy": entropy}
        if c["top"]:
            out["top_logprobs"], out["top_tokens"] = top_logprobs, top_tokens
        if c["train"]:
            out["grad_logits"] = ds.token_logprobs_backward(st["grad"], st["logits"], st["tokens"], lse,
                                                            grad_entropy=st["grad_entropy"], entropy=entropy)
        return out
    if c["op"] == "exchange":
        places, offsets = ds.expert_sort(st["experts"], c["E"])
        out = {"places": places, "offsets": offsets}
        if c["quantise"]:
            out["codes"], out["scales"] = ds.expert_gather(st["x"], places, offsets, quantise=True)
        else:
            out["rows"] = ds.expert_gather(st["x"], places, offsets)
        out["out"] = ds.expert_combine(st["y"], places, st["weights"])
        if c["train"]:
            out["grad_x"] = ds.expert_combine(st["grad_rows"], places)
            out["grad_y"], out["grad_weights"] = ds.expert_combine_backward(st["grad"], st["y"], places, offsets,
                                                                            st["weights"])
        return out
    if c["op"] == "quantise":
        codes, scales = ds.quantise_blocks(st["x"], block_rows=c["block"])
        return {"codes": codes, "scales": scales}
    return {"out": ds.expert_product(st["x"], st["x_scales"], st["w"], st["w_scales"], st["offsets"],
                                     dtype=getattr(torch, c["dtype"]))}


# ------------------------------------------------------------------ in 64 bits ---

def _round_e4m3(v):
    """v (64 bits, |v| <= 448) rounded to e4m3, ties to even."""
    _, power = torch.frexp(v)
    step = ((power.long() - 1).clamp(min=-6) + 1020 << 52).view(torch.float64)
    return torch.round(v / step) * step


def _exact_quantise(x, rows):
    codes, scales = torch.empty_like(x), torch.empty(x.shape[0], -(-x.shape[1] // rows), -(-x.shape[2] // 128),
                                                     dtype=torch.float64, device="cuda")
    for e in range(x.shape[0]):
        for j in range(scales.shape[2]):
            at = slice(128 * j, 128 * j + 128)
            size = x[e, :, at].abs().amax(-1)
            if rows > 1:
                part = torch.zeros(scales.shape[1] * rows, dtype=torch.float64, device="cuda")
                part[:size.numel()] = size
                size = part.view(-1, rows).amax(-1)
            power = torch.log2((size / 448.0).clamp(min=2.0 ** -126)).round().long()
            guess = ((power + 1023) << 52).view(torch.float64)
            # within a step of the least power of two that is enough, which comparisons then find
            s = torch.where(448.0 * guess < size, 2.0 * guess, guess)
            s = torch.where((448.0 * (0.5 * s) >= size) & (s > 2.0 ** -126), 0.5 * s, s)
            scales[e, :, j] = s
            codes[e, :, at] = _round_e4m3(x[e, :, at] / s.repeat_interleave(rows)[:x.shape[1], None])
    return codes, scales


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "logprobs":
        T, V, top = case["T"], case["V"], case["top"]
        out = {n: torch.empty(T, dtype=torch.float64, device="cuda") for n in ("logprobs", "lse", "entropy")}
        if top:
            out["top_logprobs"], out["top_tokens"] = torch.empty(T, top, dtype=torch.float64, device="cuda"), None
        if case["train"]:
            out["grad_logits"] = torch.empty(T, V, dtype=torch.float64, device="cuda")
        step = max(1, (1 << 25) // V)
        for i in range(0, T, step):
            x = st["logits"][i:i + step].double()
            z = torch.logsumexp(x, -1)
            lp = x - z[:, None]
            p = torch.exp(lp)
            H = -(p * lp).sum(-1)
            t = st["tokens"][i:i + step].long()
            hot = (t[:, None] == torch.arange(V, device="cuda")).double()
            out["lse"][i:i + step], out["entropy"][i:i + step] = z, H
            out["logprobs"][i:i + step] = (hot * lp).sum(-1)
            if top:
                out["top_logprobs"][i:i + step] = lp.topk(top, -1).values
            if case["train"]:
                g, gh = st["grad"][i:i + step].double(), st["grad_entropy"][i:i + step].double()
                g = torch.where(t >= 0, g, 0.0)
                out["grad_logits"][i:i + step] = g[:, None] * (hot - p) - gh[:, None] * p * (lp + H[:, None])
        return out
    if case["op"] == "exchange":
        T, E, k, D = (case[n] for n in ("T", "E", "k", "D"))
        chosen = st["experts"].cpu().tolist()
        by = [[] for _ in range(E)]
        for t, row in enumerate(chosen):
            for j, e in enumerate(row):
                if e >= 0:
                    by[e].append(t * k + j)
        order = torch.tensor([s for b in by for s in b], dtype=torch.int64, device="cuda")
        n = order.numel()
        t, w = order // k, st["weights"].double().view(-1)[order][:, None]
        x = torch.zeros(T * k, D, dtype=torch.float64, device="cuda")
        x[:n] = st["x"].double()[t]
        out = {"places": None, "offsets": None}
        if case["quantise"]:
            codes, scales = _exact_quantise(x[None], 1)
            out["codes"], out["scales"] = codes[0], scales[0]
        else:
            out["rows"] = x
        y = st["y"][:n].double()
        out["out"] = torch.zeros(T, D, dtype=torch.float64, device="cuda").index_add_(0, t, w * y)
        if case["train"]:
            out["grad_x"] = torch.zeros(T, D, dtype=torch.float64, device="cuda").index_add_(0, t, st["grad_rows"][:n].double())
            g = st["grad"].double()[t]
            out["grad_y"] = torch.zeros(T * k, D, dtype=torch.float64, device="cuda")
            out["grad_y"][:n] = w * g
            out["grad_weights"] = torch.zeros(T * k, dtype=torch.float64, device="cuda")
            out["grad_weights"][order] = (g * y).sum(-1)
            out["grad_weights"] = out["grad_weights"].view(T, k)
        return out
    if case["op"] == "quantise":
        codes, scales = _exact_quantise(st["x"].double(), case["block"])
        return {"codes": codes, "scales": scales}
    T, E, N, K = (case[n] for n in ("T", "E", "N", "K"))
    if 2 * T * N * K > 6e11:
        return None
    out = torch.empty(T, N, dtype=torch.float64, device="cuda")
    wide = torch.arange(K, device="cuda") // 128
    tall = torch.arange(N, device="cuda") // 128
    for e in range(E):
        a, b = st["ends"][e], st["ends"][e + 1]
        if b > a:
            x = st["x"][a:b].double() * st["x_scales"][a:b].double()[:, wide]
            out[a:b] = x @ (st["w"][e].double() * st["w_scales"][e].double()[tall][:, wide]).T
    return {"out": out}
