"""The operators behind the selections from their definitions, in torch and 64 bits, for the tests."""
import torch


def logprobs(x, tokens, top=0):
    """lse, log probability of each row's token (0 where none is given), entropy, and the top
    tokens by value, then by index."""
    x = x.double()
    V = x.shape[-1]
    m = x.amax(-1, keepdim=True)
    some = m > -torch.inf
    y = torch.where(some, x - torch.where(some, m, 0.0), -torch.inf)
    s = torch.exp(y).sum(-1, keepdim=True)
    logs = torch.where(some, torch.log(torch.where(some, s, 1.0)), 0.0)
    lp = y - logs
    p = torch.exp(lp)
    H = -torch.where(p > 0, p * lp, 0.0).sum(-1)
    t = tokens.long()
    there = (t >= 0) & (t < V)
    at = torch.where(there, t, 0)[:, None]
    given = torch.where(there, lp.gather(1, at)[:, 0], 0.0)
    order = x.sort(dim=-1, descending=True, stable=True).indices[:, :top]
    return given, (m + logs)[:, 0], H, lp.gather(1, order), order


def logprobs_gradient(x, tokens, g, h=None):
    x = x.double()
    V = x.shape[-1]
    _, lse, H, _, _ = logprobs(x, tokens)
    some = (lse > -torch.inf)[:, None]
    lp = torch.where(some, x - torch.where(some, lse[:, None], 0.0), -torch.inf)
    p = torch.exp(lp)
    t = tokens.long()
    there = (t >= 0) & (t < V)
    g = torch.where(there, g.double(), 0.0)[:, None]
    hot = (t[:, None] == torch.arange(V, device=x.device)).double()
    out = g * (hot - p)
    if h is not None:
        out = out - h.double()[:, None] * torch.where(p > 0, p * (lp + H[:, None]), 0.0)
    return torch.where(some, out, 0.0)


def sort(experts, E):
    """places and offsets of a stable counting sort, in Python's integers."""
    flat = experts.flatten().tolist()
    slots = [[] for _ in range(E)]
    for s, e in enumerate(flat):
        if 0 <= e < E:
            slots[e].append(s)
    places, offsets = [-1] * len(flat), [0]
    for run in slots:
        for j, s in enumerate(run):
            places[s] = offsets[-1] + j
        offsets.append(offsets[-1] + len(run))
    return places, offsets


def gather(x, places, rows):
    out = torch.zeros(rows, x.shape[1], dtype=x.dtype, device=x.device)
    p = places.long()
    for i in range(p.shape[1]):
        there = (p[:, i] >= 0) & (p[:, i] < rows)
        out[p[there, i]] = x[there]
    return out


def combine(y, places, weights=None):
    """(sums, sums of sizes) in 64 bits."""
    y, p = y.double(), places.long()
    out = torch.zeros(p.shape[0], y.shape[1], dtype=torch.float64, device=y.device)
    size = out.clone()
    for i in range(p.shape[1]):
        there = (p[:, i] >= 0) & (p[:, i] < y.shape[0])
        w = 1.0 if weights is None else weights.double()[there, i, None]
        v = w * y[p[there, i]]
        out[there] += v
        size[there] += v.abs()
    return out, size


def scale_of(top):
    """The least power of two >= 2^-126 with top <= 448 of it, for a Python number."""
    s = 2.0 ** -126
    while top > 448.0 * s:
        s *= 2.0
    return s


def round_e4m3(v):
    """Numbers up to 448 in size to e4m3: 4 significant bits down to 2^-6, steps of 2^-9 below; ties
    to even."""
    v = v.double()
    _, power = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (power - 1).clamp(min=-6) - 3)
    step = torch.exp2(torch.log2(step).round())
    return torch.round(v / step) * step


def quantise(x, block_rows):
    """(codes as numbers, scales) of x (E, N, K), in 64 bits."""
    x = x.double()
    E, N, K = x.shape
    nb, kb = -(-N // block_rows), -(-K // 128)
    scales = torch.zeros(E, nb, kb, dtype=torch.float64, device=x.device)
    codes = torch.zeros_like(x)
    for e in range(E):
        for i in range(nb):
            for j in range(kb):
                at = (e, slice(i * block_rows, (i + 1) * block_rows), slice(128 * j, 128 * j + 128))
                s = scale_of(float(x[at].abs().max()))
                scales[e, i, j] = s
                codes[at] = round_e4m3(x[at] / s)
    return codes, scales


def product(x, xs, w, ws, offsets):
    """(rows, N) in 64 bits, and the sums of the products' sizes."""
    T, K = x.shape
    E, N, _ = w.shape
    wide, tall = torch.arange(K, device=x.device) // 128, torch.arange(N, device=x.device) // 128
    out = torch.zeros(T, N, dtype=torch.float64, device=x.device)
    size = out.clone()
    for e in range(E):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if b > a:
            v = x[a:b].double() * xs[a:b].double()[:, wide]
            m = w[e].double() * ws[e].double()[tall][:, wide]
            out[a:b] = v @ m.T
            size[a:b] = v.abs() @ m.abs().T
    return out, size
