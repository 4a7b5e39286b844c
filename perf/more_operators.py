"""Timing cases of the operators between the products of a decode step and behind its head: keys and values rotated,
quantised and written into a paged cache, read back from it, the attention of new tokens over it, and the choice of
the next tokens from the logits.  ``run`` computes them with elementary torch operations, or, with ``own`` set, with
this package."""
import math

import torch

own = False

BASE = 500000.0     # of the rotation's angles
PLANTED = 6.0       # some channels of the keys are that much larger


def _heads(q, kv, dim):
    return dict(q_heads=q, kv_heads=kv, dim=dim)


H70, H9, H8 = _heads(64, 8, 128), _heads(16, 8, 256), _heads(32, 8, 128)


def listed():
    return [
        # one token of one request behind the q|k|v product of a 70B-shaped layer: latency alone
        dict(name="write, 1 token", op="write", b=1, page=16, fmt="int8", rot=128, interleaved=False, **H70),
        # a packed prompt of a 9B-shaped layer, quantised as it is written, an odd number of tokens
        dict(name="write, 2047 tokens", op="write", b=2047, page=64, fmt="int8", rot=256, interleaved=False, **H9),
        # a prompt's keys and values for a program that goes on with them in fp16
        dict(name="read, 16381 tokens", op="read", b=16381, page=64, fmt="int8", **H70),
        # the tokens of a short prefix that two requests share
        dict(name="read, 133 tokens", op="read", b=133, page=16, fmt="int8", **H8),
        # one request early on
        dict(name="attend, 1 of 509", op="attend", b=1, L=509, page=16, fmt="int8", softcap=0.0, window=0, **H8),
        # one request with a long document: the cache's length is all there is to split
        dict(name="attend, 1 of 131072", op="attend", b=1, L=131072, page=64, fmt="int8", softcap=0.0, window=0, **H70),
        # a decode batch of requests of every length, one of them not begun
        dict(name="attend, 64 of up to 8192", op="attend", b=64, L=8192, page=64, fmt="int8", softcap=0.0, window=0,
             **H70),
        # a 9B-shaped layer that sees a window and bounds its scores, over an fp16 cache
        dict(name="attend window, 37 of up to 6001", op="attend", b=37, L=6001, page=48, fmt="fp16", softcap=50.0,
             window=4096, **H9),
        # a decode step's part between q|k|v and o: write the new tokens, attend, read the written rows back
        dict(name="step, 16 of up to 2048", op="step", b=16, L=2048, page=16, fmt="int8", softcap=0.0, window=0,
             rot=128, interleaved=False, **H70),
        # the next token of one request, every filter on
        dict(name="sample, 1 of 128256", op="sample", b=1, N=128256, k=True, p=True, m=True, T=True),
        # a batch that draws from the whole vocabulary
        dict(name="sample all, 61 of 128256", op="sample", b=61, N=128256, k=False, p=False, m=False, T=True),
        # the largest vocabulary for a large decode batch
        dict(name="sample, 256 of 256000", op="sample", b=256, N=256000, k=True, p=True, m=False, T=True),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["write", "read", "attend", "attend", "step", "sample", "sample"])
    if op == "sample":
        b = _log(rng, 1, 256)
        on = [rng.random() < 0.6 for _ in range(4)]
        return dict(op=op, b=b, N=_log(rng, 100, 256000), k=on[0], p=on[1], m=on[2], T=on[3])
    heads = rng.choice([H70, H9, H8, _heads(12, 12, 64), _heads(20, 5, 96), _heads(16, 1, 128), _heads(40, 1, 64),
                        _heads(28, 4, 128), _heads(6, 2, 80)])
    case = dict(op=op, page=rng.choice([16, 32, 48, 64, 128, 256]), fmt=rng.choice(["int8", "int8", "fp16"]), **heads)
    wide = heads["kv_heads"] * heads["dim"] * (2 if case["fmt"] == "fp16" else 1)
    if op == "read":
        return dict(case, b=min(_log(rng, 1, 16381), 16381 * 1024 // wide))
    if op in ("write", "step"):
        case.update(rot=rng.choice([heads["dim"], heads["dim"], heads["dim"] // 32 * 16]),
                    interleaved=rng.random() < 0.3)
    if op == "write":
        return dict(case, b=_log(rng, 1, 2047))
    case.update(b=_log(rng, 1, 256), softcap=rng.choice([0.0, 0.0, 50.0]))
    case["L"] = min(_log(rng, 1, 131072), 64 * 8192 * 1024 // (case["b"] * wide))
    case["window"] = rng.choice([0, 0, _log(rng, 1, 8192)])
    return case


def _lens(case):
    """How many tokens each row sees: every length up to L, one row empty and one with a single token."""
    b, L = case["b"], case["L"]
    lens = [1 + int((L - 1) * ((r + 1) * 0.6180339887498949 % 1.0)) for r in range(b)]
    lens[0] = L
    if b >= 6:
        lens[3], lens[5] = 0, 1
    return lens


def _seen(case):
    """How many of them its window leaves."""
    return [min(n, case["window"] or n) for n in _lens(case)]


def _size(case):
    return 1 if case["fmt"] == "int8" else 2


# ----------------------------------------------------------------- inputs

def _pool(g, n_pages, case):
    """A cache: fp16 values, or codes + 128 as INT8 weights lie in device memory with a scale for each token and head."""
    shape = (n_pages, case["kv_heads"], case["page"], case["dim"])
    out = {}
    for name in ("k", "v"):
        fmt8 = case["fmt"] == "int8"
        t = torch.empty(shape, dtype=torch.uint8 if fmt8 else torch.float16, device="cuda")
        scale = torch.empty(shape[:3], device="cuda") if fmt8 else None
        some = max(1, (1 << 26) // (shape[1] * shape[2] * shape[3]))
        for i in range(0, n_pages, some):
            x = torch.randn(t[i:i + some].shape, generator=g, device="cuda")
            if name == "k":
                x[..., ::37] *= PLANTED
            if fmt8:
                step = x.abs().amax(-1) / 127
                scale[i:i + some] = step
                t[i:i + some] = (x / step[..., None]).round_() + 128
            else:
                t[i:i + some] = x
        out[name], out[name + "_scale"] = t, scale
    return out


def _rope(n_pos, rot):
    """cos | sin of every position's angles, taken in 64 bits."""
    turn = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    a = torch.arange(n_pos, dtype=torch.float64, device="cuda")[:, None] * turn
    return torch.cat([a.cos(), a.sin()], 1).float()


def _tables(g, case, s):
    """Pages of a shuffled pool for every row, -1 behind the last, and the row's new token's slot and position."""
    lens, page, b = _lens(case), case["page"], case["b"]
    need = [-(-n // page) for n in lens]
    n_pages = sum(need) + 3
    order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    pages = torch.full((b, max(need)), -1, dtype=torch.int32)
    first = 0
    for r, n in enumerate(need):
        pages[r, :n] = torch.arange(first, first + n)
        first += n
    pages = pages.cuda()
    s["pages"] = torch.where(pages >= 0, order[pages.clamp(min=0).long()], pages)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["n_pages"], s["longest"] = n_pages, max(lens)
    at = (s["lens"].long() - 1).clamp(min=0)
    slot = s["pages"].long().gather(1, (at // page)[:, None])[:, 0] * page + at % page
    s["slots"] = torch.where(s["lens"] > 0, slot, torch.full_like(slot, -1)).to(torch.int32)
    s["spare"] = order[-1].long() * page        # of a page that no row has
    s["pos"] = at.to(torch.int32)


def _logits(g, case, s):
    b, N = case["b"], case["N"]
    x = torch.randn(b, -(-N // 8) * 8, generator=g, device="cuda") * 2.5 - 1.0
    # a handful of tokens that the context asks for
    some = torch.randint(0, N, (b, 24), generator=g, device="cuda")
    x.scatter_add_(1, some, 3.0 + 9.0 * torch.rand(b, 24, generator=g, device="cuda"))
    # tokens that a grammar rules out
    x[::2, 5:N:97] = -math.inf
    s["logits"] = x.half()

    def pick(values):
        v = torch.tensor(values, device="cuda")
        return v[torch.randint(0, len(values), (b,), generator=g, device="cuda")]

    s["T"] = pick([0.0, 0.6, 0.7, 1.0, 1.0, 1.3]) if case["T"] else None
    s["top_k"] = pick([0, 1, 20, 40, 1000]).to(torch.int32) if case["k"] else None
    s["top_p"] = pick([0.5, 0.9, 0.95, 1.0]) if case["p"] else None
    s["min_p"] = pick([0.0, 0.02, 0.1]) if case["m"] else None
    s["u"] = torch.rand(b, generator=g, device="cuda")
    s["token"] = torch.empty(b, dtype=torch.int32, device="cuda")
    s["prob"] = torch.empty(b, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, b = case["op"], case["b"]
    s = dict(case)
    half = dict(dtype=torch.float16, device="cuda")
    if op == "sample":
        _logits(g, case, s)
        return s
    Hq, Hk, D, page = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    if op in ("attend", "step"):
        _tables(g, case, s)
    else:
        # one prompt's tokens in the order of a shuffled pool's pages, the last page not full
        s["n_pages"] = -(-b // page) + 1
        at = torch.arange(b, device="cuda")
        order = torch.randperm(s["n_pages"], generator=g, device="cuda")
        s["slots"] = (order[at // page] * page + at % page).to(torch.int32)
        s["pos"] = (at + seed % 64).to(torch.int32)
    s.update(_pool(g, s["n_pages"], case))
    if op in ("write", "step"):
        # q, k and v side by side in one row, as the stacked product writes them
        x = torch.randn(b, (Hq + 2 * Hk) * D, generator=g, device="cuda")
        x[:, Hq * D:(Hq + Hk) * D:37] *= PLANTED
        s["qkv"] = x.half()
        s["rope"] = _rope(s["longest"] if op == "step" else b + 64, case["rot"])
        s["q_out"] = torch.empty(b, Hq * D, **half)
    if op == "attend":
        s["q"] = torch.randn(b, Hq * D, generator=g, device="cuda").half()
    if op in ("attend", "step"):
        s["y"] = torch.empty(b, Hq * D, **half)
    # the rows to read back: of a prompt's pages all, of a step those just written
    s["back"] = s["slots"] if op != "write" else torch.arange(s["n_pages"] * page, device="cuda", dtype=torch.int32)
    s["k_out"] = torch.empty(len(s["back"]), Hk * D, **half)
    s["v_out"] = torch.empty(len(s["back"]), Hk * D, **half)
    return s


# -------------------------------------------------------- the plain forms

def _rotate(x, s):
    """x [b, heads, dim] turned by its row's angles: pairs a half apart, or next to each other."""
    rot = s["rot"]
    cs = s["rope"][s["pos"].long()][:, None]
    c, sn = cs[..., :rot // 2], cs[..., rot // 2:]
    part, rest = x[..., :rot], x[..., rot:]
    if s["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([a * c - b * sn, b * c + a * sn], -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        turned = torch.cat([a * c - b * sn, b * c + a * sn], -1)
    return torch.cat([turned, rest], -1)


def _split(s):
    Hq, Hk, D = s["q_heads"], s["kv_heads"], s["dim"]
    x = s["qkv"].float().view(s["b"], Hq + 2 * Hk, D)
    return _rotate(x[:, :Hq], s), _rotate(x[:, Hq:Hq + Hk], s), x[:, Hq + Hk:]


def _plain_write(s):
    q, k, v = _split(s)
    slots = s["slots"].long()
    if s["op"] == "step":       # rows that have not begun write where nothing is read
        slots = torch.where(slots >= 0, slots, s["spare"])
    at, off = slots // s["page"], slots % s["page"]
    for name, x in (("k", k), ("v", v)):
        if s["fmt"] == "int8":
            scale = x.abs().amax(-1) / 127
            safe = torch.where(scale > 0, scale, torch.ones_like(scale))
            s[name][at, :, off] = ((x / safe[..., None]).round() + 128).to(torch.uint8)
            s[name + "_scale"][at, :, off] = scale
        else:
            s[name][at, :, off] = x.half()
    return q.half().flatten(1)


def _plain_read(s):
    slots = s["back"].long()
    on, slots = slots >= 0, slots.clamp(min=0)
    at, off = slots // s["page"], slots % s["page"]
    got = []
    for name in ("k", "v"):
        x = s[name][at, :, off].float()
        if s["fmt"] == "int8":
            x = (x - 128) * s[name + "_scale"][at, :, off][..., None]
        got.append(torch.where(on[:, None, None], x, torch.zeros_like(x)).half().flatten(1))
    return got


def _gather(s, name):
    """Every row's tokens [b, kv_heads, tokens, dim], whatever stands behind its last."""
    t = s[name][s["pages"].clamp(min=0).long()]
    b, W, Hk, page = t.shape[:4]
    t = t.transpose(1, 2).reshape(b, Hk, W * page, -1).float()
    if s["fmt"] == "int8":
        scale = s[name + "_scale"][s["pages"].clamp(min=0).long()].transpose(1, 2).reshape(b, Hk, W * page, 1)
        t = (t - 128) * scale
    return t


def _plain_attend(q, s):
    b, Hq, Hk, D = s["b"], s["q_heads"], s["kv_heads"], s["dim"]
    q = q.float().view(b, Hk, Hq // Hk, D)
    scores = torch.matmul(q, _gather(s, "k").transpose(2, 3).contiguous()) * D ** -0.5
    if s["softcap"]:
        scores = s["softcap"] * torch.tanh(scores / s["softcap"])
    t = torch.arange(scores.shape[-1], device=q.device)
    n = s["lens"].long()[:, None]
    seen = (t < n) & (t >= n - s["window"]) if s["window"] else t < n
    seen = seen[:, None, None]
    scores = torch.where(seen, scores, torch.full_like(scores, -math.inf))
    top = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - torch.where(top > -math.inf, top, torch.zeros_like(top)))
    total = e.sum(-1, keepdim=True)
    p = e / torch.where(total > 0, total, torch.ones_like(total))
    return torch.matmul(p, _gather(s, "v")).half().view(b, Hq * D)


def _plain_sample(s):
    x = s["logits"][:, :s["N"]].double()
    b, N = x.shape
    x, order = torch.sort(x, descending=True, stable=True)
    first = torch.arange(N, device=x.device) == 0
    T = s["T"].double()[:, None] if s["T"] is not None else torch.ones(b, 1, dtype=torch.float64, device=x.device)
    w = torch.exp((x - x[:, :1]) / torch.where(T > 0, T, torch.ones_like(T)))
    keep = (x > -math.inf) & ((T > 0) | first)
    if s["top_k"] is not None:
        k = s["top_k"].long()[:, None]
        keep &= (torch.arange(N, device=x.device) < k) | (k <= 0)
    if s["min_p"] is not None:
        keep &= w >= s["min_p"].double()[:, None]
    w = torch.where(keep, w, torch.zeros_like(w))
    if s["top_p"] is not None:
        p = s["top_p"].double()[:, None]
        before = torch.cumsum(w, 1) - w
        keep &= (before < p * w.sum(1, keepdim=True)) | (p >= 1) | first
        w = torch.where(keep, w, torch.zeros_like(w))
    cum = torch.cumsum(w, 1)
    total = cum[:, -1:]
    at = (cum <= s["u"].double()[:, None] * total).sum(1, keepdim=True)
    at = torch.minimum(at, keep.sum(1, keepdim=True) - 1)
    token = order.gather(1, at)[:, 0].to(torch.int32)
    return {"token": token, "prob": (w.gather(1, at) / total)[:, 0].float()}


# ------------------------------------------------------- this package's

def _cache(s):
    """The handle that a program keeps for its cache, made on the first pass."""
    from weight_only_quantized_quantize_amd import woq
    if "cache" not in s:
        s["cache"] = woq.DeviceCache(s["k"], s["v"], s["k_scale"], s["v_scale"])
    return woq, s["cache"].desc


def _own_write(s):
    woq, cache = _cache(s)
    n, m = s["q_heads"] * s["dim"], s["kv_heads"] * s["dim"]
    x = s["qkv"]
    woq.woq_cache_write(cache, x[:, n:n + m], x[:, n + m:], s["slots"], q=x[:, :n], q_out=s["q_out"], rope=s["rope"],
                        pos=s["pos"], interleaved=s["interleaved"])


def _own_read(s):
    woq, cache = _cache(s)
    woq.woq_cache_read(cache, s["back"], s["k_out"], s["v_out"])


def _own_attend(q, s):
    woq, cache = _cache(s)
    if "work" not in s:
        n = woq.woq_attn_decode_workspace(cache, s["q_heads"], s["b"])
        s["work"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    woq.woq_attn_decode(cache, q, s["pages"], s["lens"], s["y"], s["work"], scale=s["dim"] ** -0.5,
                        softcap=s["softcap"], window=s["window"])


def _own_sample(s):
    from weight_only_quantized_quantize_amd import woq
    woq.woq_sample(s["logits"], s["u"], s["token"], temperature=s["T"], top_k=s["top_k"], top_p=s["top_p"],
                   min_p=s["min_p"], prob=s["prob"], N=s["N"])
    return {"token": s["token"], "prob": s["prob"]}


def run(s):
    op = s["op"]
    if op == "sample":
        return _own_sample(s) if own else _plain_sample(s)
    if op == "attend":
        if not own:
            return {"y": _plain_attend(s["q"], s)}
        _own_attend(s["q"], s)
        return {"y": s["y"]}
    if own:
        got = {}
        if op != "read":
            _own_write(s)
            got["q"] = s["q_out"]
        if op == "step":
            _own_attend(s["q_out"], s)
            got["y"] = s["y"]
        _own_read(s)
        return dict(got, k=s["k_out"], v=s["v_out"])
    got = {}
    if op != "read":
        got["q"] = _plain_write(s)
    if op == "step":
        got["y"] = _plain_attend(got["q"], s)
    got["k"], got["v"] = _plain_read(s)
    return got


def work(case):
    op, b = case["op"], case["b"]
    if op == "sample":
        return {"bytes": 2 * b * case["N"] + 28 * b, "flops": 2 * b * case["N"]}
    Hq, Hk, D, page = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    row = Hk * (D * _size(case) + (4 if case["fmt"] == "int8" else 0))      # of the keys or the values of a token
    nbytes = flops = 0
    if op in ("write", "step"):
        nbytes += 2 * b * (Hq + 2 * Hk) * D + 2 * b * Hq * D + 2 * b * row + b * (8 + 4 * case["rot"])
        flops += b * (6 * Hq + 10 * Hk) * D
    if op in ("attend", "step"):
        seen = sum(_seen(case))
        nbytes += 2 * seen * row + 4 * b * Hq * D + 4 * seen // page + 4 * b
        flops += 4 * seen * Hq * D
    if op in ("write", "read", "step"):
        n = b if op != "write" else (-(-b // page) + 1) * page
        nbytes += n * (4 + 2 * row + 4 * Hk * D)
        flops += 4 * n * Hk * D
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------ the definitions, in 64 bits

def _exact_rows(s):
    """q, k and v of the new tokens in 64 bits: each pair (a, b) turned by its angle, as complex numbers are."""
    Hq, Hk, D, rot, b = s["q_heads"], s["kv_heads"], s["dim"], s["rot"], s["b"]
    x = s["qkv"].double().reshape(b, Hq + 2 * Hk, D).clone()
    table = s["rope"].double()[s["pos"].long()]
    turn = torch.complex(table[:, :rot // 2], table[:, rot // 2:])[:, None]
    if s["interleaved"]:
        i, j = torch.arange(0, rot, 2), torch.arange(1, rot, 2)
    else:
        i, j = torch.arange(0, rot // 2), torch.arange(rot // 2, rot)
    i, j = i.cuda(), j.cuda()
    z = torch.complex(x[:, :Hq + Hk, i], x[:, :Hq + Hk, j]) * turn
    x[:, :Hq + Hk, i], x[:, :Hq + Hk, j] = z.real, z.imag
    return x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]


def _stored(x, s):
    """What a cache holds of rows x: fp16 values, or the nearest of 255 steps."""
    if s["fmt"] != "int8":
        return x.half().double()
    step = x.abs().max(-1, keepdim=True).values / 127
    return torch.round(x / step) * step


def _exact_cache(s, name, at, off):
    x = s[name][at, :, off].double()
    return x if s["fmt"] != "int8" else (x - 128) * s[name + "_scale"][at, :, off].double()[..., None]


def exact(case, seed):
    s = prepare(case, seed)
    op, b = case["op"], case["b"]
    if op == "sample":
        return _exact_sample(s)
    Hq, Hk, D, page = case["q_heads"], case["kv_heads"], case["dim"], case["page"]
    got = {}
    if op in ("write", "step"):
        q, k, v = _exact_rows(s)
        got["q"] = q.flatten(1)
        new = {"k": _stored(k, s), "v": _stored(v, s)}
        s["q"] = q
    if op in ("attend", "step"):
        y = torch.zeros(b, Hq, D, dtype=torch.float64, device="cuda")
        for r, n in enumerate(_lens(case)):
            if not n:
                continue
            t = torch.arange(max(0, n - case["window"]) if case["window"] else 0, n, device="cuda")
            at, off = s["pages"][r].long()[t // page], t % page
            K, V = _exact_cache(s, "k", at, off), _exact_cache(s, "v", at, off)
            if op == "step":
                K[-1], V[-1] = new["k"][r], new["v"][r]
            q = s["q"].double().reshape(b, Hk, Hq // Hk, D)[r]
            z = torch.matmul(q, K.permute(1, 2, 0).contiguous()) / math.sqrt(D)
            if case["softcap"]:
                z = torch.tanh(z / case["softcap"]) * case["softcap"]
            p = torch.softmax(z, -1)
            y[r] = torch.matmul(p, V.permute(1, 0, 2).contiguous()).reshape(Hq, D)
        got["y"] = y.flatten(1)
    if op == "attend":
        return got
    for name in ("k", "v"):
        n = s["n_pages"] * page
        every = torch.arange(n, device="cuda")
        if op == "read":
            slots = s["slots"].long()
            got[name] = _exact_cache(s, name, slots // page, slots % page).flatten(1)
            continue
        if op == "write":
            x = _exact_cache(s, name, every // page, every % page)
            x[s["slots"].long()] = new[name]
        else:
            x = torch.where((s["slots"] >= 0)[:, None, None], new[name], torch.zeros_like(new[name]))
        got[name] = x.flatten(1)
    return got


def _exact_sample(s):
    """Row by row over its distinct logits, from the largest down: how many there are, what each weighs, how many stay."""
    tokens, probs = [], []
    for r in range(s["b"]):
        x = s["logits"][r, :s["N"]].double()
        value, count = torch.unique(x[x > -math.inf], return_counts=True)
        value, count = value.flip(0), count.flip(0)
        T = 1.0 if s["T"] is None else float(s["T"][r])
        k = 0 if s["top_k"] is None else int(s["top_k"][r])
        m = 0.0 if s["min_p"] is None else float(s["min_p"][r])
        p = 1.0 if s["top_p"] is None else float(s["top_p"][r])
        if not T > 0:
            T, k = 1.0, 1
        w = torch.exp((value - value[0]) / T)
        left = count.clone()
        if k > 0:
            left = torch.minimum(count, (k - (count.cumsum(0) - count)).clamp(min=0))
        left = torch.where(w >= m, left, torch.zeros_like(left))
        mass = w * left
        if p < 1:
            need = p * mass.sum() - (mass.cumsum(0) - mass)     # what the tokens above leave to reach
            left = torch.minimum(left, torch.ceil(need / w).clamp(min=0).long())
            left[0] = left[0].clamp(min=1)
            mass = w * left
        total = mass.sum()
        t = float(s["u"][r].double() * total)
        end = mass.cumsum(0)
        i = min(int((end <= t).sum()), int((left > 0).sum()) - 1)
        j = min(max(int((t - float(end[i] - mass[i])) // float(w[i])), 0), int(left[i]) - 1)
        tokens.append(torch.nonzero(x == value[i])[j, 0])
        probs.append(w[i] / total)
    return {"token": torch.stack(tokens).to(torch.int32), "prob": torch.stack(probs)}
