"""Timing cases of the operators around a quantised linear: the residual addition and RMS norm with fp16 and 8-bit
outputs, the product of INT8 weights with those 8-bit rows, and the low-rank adapters added beside a shared
projection.  ``run`` computes them with elementary torch operations, or, with ``own`` set, with this package."""
import math

import torch

own = False

EPS = 1e-6
PLANTED = 20.0      # the outlier channels of hidden states are that much larger


def listed():
    return [
        # one token of one request between two products of a 70B-shaped layer: latency alone
        dict(name="norm, 1 token", op="norm", b=1, K=8192, residual=True, fp16=True, int8=False),
        # a ragged decode batch whose next product takes 8-bit rows (9B-shaped hidden width)
        dict(name="norm int8, 37 tokens", op="norm", b=37, K=3584, residual=True, fp16=False, int8=True),
        # a packed prompt of a 70B-shaped stack, both outputs (adapters read the fp16 one)
        dict(name="norm both, 4096 tokens", op="norm", b=4096, K=8192, residual=True, fp16=True, int8=True),
        # q|k|v of a 9B-shaped layer for one token: the weights are read once
        dict(name="product, 1 token", op="product", b=1, N=8192, K=3584),
        # gate|up of that layer for a large decode batch
        dict(name="product, 61 tokens", op="product", b=61, N=28672, K=3584),
        # down for a short prompt: a long row
        dict(name="product, 509 tokens", op="product", b=509, N=3584, K=14336),
        # gate|up for a long packed prompt: bound by the matrix cores
        dict(name="product, 4095 tokens", op="product", b=4095, N=28672, K=3584),
        # one request with its adapter beside a 70B-shaped o
        dict(name="adapters, 1 token", op="adapters", b=1, K=8192, N=8192, segments=1, R=16, count=8),
        # a decode batch in which every request has an adapter of its own, beside q|k|v
        dict(name="adapters, 64 tokens", op="adapters", b=64, K=8192, N=10240, segments=3, R=16, count=64),
        # packed prompts of several requests beside gate|up
        dict(name="adapters, 3001 tokens", op="adapters", b=3001, K=3584, N=28672, segments=2, R=64, count=8),
        # norm, 8-bit product and adapters in a row: q|k|v of a 9B-shaped layer, decode and prompt
        dict(name="all three, 8 tokens", op="layer", b=8, K=3584, N=8192, segments=3, R=16, count=4),
        dict(name="all three, 1021 tokens", op="layer", b=1021, K=3584, N=8192, segments=3, R=16, count=4),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["norm", "product", "adapters", "layer"])
    b = _log(rng, 1, 4096)
    if op == "norm":
        K = min(_log(rng, 256, 16384), 4096 * 8192 // b)
        fp16, int8 = rng.choice([(True, False), (False, True), (True, True)])
        return dict(op=op, b=b, K=K, residual=rng.random() < 0.7, fp16=fp16, int8=int8)
    N = min(_log(rng, 64, 28672), 3001 * 28672 // b)
    K = min(_log(rng, 128, 14336), 4095 * 28672 * 3584 // (b * N))
    if op == "product":
        return dict(op=op, b=b, N=N, K=K)
    R, segments = 8 * rng.randint(1, 8), rng.randint(1, 3)
    return dict(op=op, b=b, K=K, N=N, segments=segments, R=R, count=_log(rng, 1, 64 if b <= 64 else 8))


def _up(n, m):
    return -(-n // m) * m


def _ends(case):
    """Where the segments of N end: the first takes about half, as q beside k and v does."""
    S, N = case["segments"], case["N"]
    return {1: [N], 2: [N // 2, N], 3: [N // 2, N // 2 + N // 4, N]}[S]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, b, K = case["op"], case["b"], case["K"]

    def normal(*shape, std=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * std

    s = {"op": op, "b": b, "K": K}
    half = dict(dtype=torch.float16, device="cuda")
    if op != "product":
        # hidden states: a hundredth of the channels is far larger than the rest
        x = normal(b, _up(K, 8))
        x[:, torch.randperm(K, generator=g, device="cuda")[:-(-K // 100)]] *= PLANTED
        s["x"] = x.half()
    if op in ("norm", "layer"):
        s["res"] = normal(b, _up(K, 8), std=2.0).half() if case.get("residual", True) else None
        s["weight"] = (1.0 + normal(K, std=0.1)).half()
        s["fp16"], s["int8"] = case.get("fp16", True), case.get("int8", True)
        # what a program keeps for the results
        s["sum"] = torch.empty(b, _up(K, 8), **half) if s["res"] is not None else None
        s["y"] = torch.empty(b, _up(K, 8), **half) if s["fp16"] else None
        s["q"] = torch.empty(b, _up(K, 16), dtype=torch.int8, device="cuda") if s["int8"] else None
        s["q_scale"] = torch.empty(b, device="cuda") if s["int8"] else None
        s["deq"] = torch.empty(b, K, **half) if s["int8"] else None
    if op == "product":
        x = normal(b, K)
        s["q"] = torch.zeros(b, _up(K, 16), dtype=torch.int8, device="cuda")
        s["q_scale"] = x.abs().amax(1) / 127
        s["q"][:, :K] = (x / s["q_scale"][:, None]).round()
    if op in ("product", "layer"):
        # the INT8 weight as it lies in device memory: code + 128, rows padded to 64 columns, 4 rows
        N = case["N"]
        W = normal(N, K, std=0.02)
        scale = W.abs().max() / 127
        s["codes"] = torch.full((_up(N, 4), _up(K, 64)), 128, dtype=torch.uint8, device="cuda")
        s["codes"][:N, :K] = (W / scale).round() + 128
        s["w_scale"], s["N"] = float(scale), N
        s["out"] = torch.empty(b, N, **half)
    if op in ("adapters", "layer"):
        N, S, R, n = case["N"], case["segments"], case["R"], case["count"]
        s["N"], s["R"], s["ends"] = N, R, _ends(case)
        s["A"] = torch.zeros(n, S * R, _up(K, 8), **half)
        s["A"][:, :, :K] = normal(n, S * R, K, std=K ** -0.5)
        s["B"] = normal(n, N, R, std=0.05).half()
        s["scale"] = 0.5 + torch.rand(n, generator=g, device="cuda")
        if b <= 64:     # decode: a row is a request
            ids = torch.arange(b, device="cuda") % n
            ids = ids[torch.randperm(b, generator=g, device="cuda")]
        else:           # packed prompts: requests of different lengths, one of them without an adapter
            cuts = torch.randint(1, b, (2 * n,), generator=g, device="cuda").sort().values
            ids = (torch.searchsorted(cuts, torch.arange(b, device="cuda"), right=True) * 5 + 3) % (n + 1) - 1
        s["ids"] = ids.to(torch.int32)
        if op == "adapters":
            s["base"] = normal(b, N).half()
        s["with_adapters"] = torch.empty(b, N, **half)
    return s


def _norm(s):
    x = s["x"][:, :s["K"]].float()
    if s["res"] is not None:
        x = x + s["res"][:, :s["K"]].float()
    v = x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS) * s["weight"].float()
    scale = v.abs().amax(1) / 127
    safe = torch.where(scale > 0, scale, torch.ones_like(scale))
    return x.half(), v.half(), (v / safe[:, None]).round(), scale


def _product(codes, scale, s):
    w = s["codes"][:s["N"], :s["K"]].float() - 128
    return ((codes @ w.t()) * (scale[:, None] * s["w_scale"])).half()


def _adapters(x, base, s):
    n, N, R = s["B"].shape
    S = len(s["ends"])
    b = x.shape[0]
    dev = x.device
    rows = torch.arange(b, device=dev)
    ids = s["ids"].long()
    on = (ids >= 0) & (ids < n)
    at = ids.clamp(0, n - 1)
    seg = torch.searchsorted(torch.tensor(s["ends"], device=dev), torch.arange(N, device=dev), right=True)
    if b <= 64:      # each row's own adapter, gathered
        h = torch.matmul(s["A"][at, :, :s["K"]].float(), x.float()[:, :, None]).view(b, S, R)
        delta = (s["B"][at].float() * h[:, seg]).sum(2)
    else:            # every adapter over all rows; the others' parts are then left out
        A = s["A"][:, :, :s["K"]].float()
        h = (x.float() @ A.view(n * S * R, -1).t()).view(b, n, S * R)[rows, at]
        z = torch.zeros(b, n, S * R, device=dev)
        z[rows, at] = h
        mask = (seg[:, None] == torch.arange(S, device=dev)).float()
        wide = s["B"].float().permute(1, 0, 2)[:, :, None, :] * mask[:, None, :, None]
        delta = z.view(b, -1) @ wide.reshape(N, -1).t()
    delta = torch.where(on[:, None], delta * s["scale"][at][:, None], torch.zeros_like(delta))
    return (base.float() + delta).half()


def _int8_weight(s):
    """The handle that a program keeps for its weight, made on the first pass."""
    from weight_only_quantized_quantize_amd import woq
    w = woq.Int8W()
    w.codes, w.N, w.K, w.nseg = s["codes"].data_ptr(), s["N"], s["K"], 1
    w.seg_end[0], w.seg_scale[0] = s["N"], s["w_scale"]
    return w


def _run_own(s):
    from weight_only_quantized_quantize_amd import woq
    op = s["op"]
    if op in ("product", "layer") and "w8" not in s:
        s["w8"] = _int8_weight(s)
    if op in ("adapters", "layer") and "lora" not in s:
        s["lora"] = woq.DeviceLora(s["A"], s["B"], s["scale"], K=s["K"], segments=s["ends"])
        s["work"] = torch.empty(woq.woq_lora_workspace(s["lora"].desc, s["b"]), dtype=torch.uint8, device="cuda")
    if op in ("norm", "layer"):
        woq.woq_add_rmsnorm(s["x"], s["weight"], EPS, res=s["res"], sum_out=s["sum"], y=s["y"], q=s["q"],
                            q_scale=s["q_scale"])
    if op in ("product", "layer"):
        woq.woq_qgemm_int8_a8(s["w8"], s["q"], s["q_scale"], s["out"])
    if op == "product":
        return {"y": s["out"]}
    if op == "adapters":
        woq.woq_lora_add(s["lora"].desc, s["x"], s["ids"], s["base"], s["with_adapters"], s["work"])
        return {"y": s["with_adapters"]}
    K = s["K"]
    if op == "layer":
        woq.woq_lora_add(s["lora"].desc, s["y"], s["ids"], s["out"], s["with_adapters"], s["work"])
        return {"sum": s["sum"][:, :K], "normed": s["y"][:, :K], "y": s["with_adapters"]}
    got = {}
    if s["sum"] is not None:
        got["sum"] = s["sum"][:, :K]
    if s["fp16"]:
        got["y"] = s["y"][:, :K]
    if s["int8"]:
        got["codes"] = torch.mul(s["q"][:, :K], s["q_scale"][:, None], out=s["deq"])
        got["scale"] = s["q_scale"]
    return got


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "product":
        return {"y": _product(s["q"][:, :s["K"]].float(), s["q_scale"], s)}
    if op == "adapters":
        return {"y": _adapters(s["x"][:, :s["K"]], s["base"], s)}
    total, y, codes, scale = _norm(s)
    if op == "layer":
        return {"sum": total, "normed": y, "y": _adapters(y, _product(codes, scale, s), s)}
    got = {}
    if s["res"] is not None:
        got["sum"] = total
    if s["fp16"]:
        got["y"] = y
    if s["int8"]:
        got["codes"] = (codes * scale[:, None]).half()
        got["scale"] = scale
    return got


def work(case):
    op, b, K = case["op"], case["b"], case["K"]
    nbytes = flops = 0
    if op in ("norm", "layer"):
        per = 2 + (4 if case.get("residual", True) else 0) + 2 * case.get("fp16", True)
        per += case.get("int8", True) and op == "norm"
        nbytes += b * K * per + 2 * K
        flops += 6 * b * K
    if op in ("product", "layer"):
        nbytes += case["N"] * K + (b * K + 4 * b + 2 * b * case["N"] if op == "product" else 0)
        flops += 2 * b * case["N"] * K
    if op in ("adapters", "layer"):
        used, ranks, N = min(b, case["count"]), case["segments"] * case["R"], case["N"]
        nbytes += 2 * used * (ranks * K + N * case["R"]) + 2 * b * N + 4 * b
        nbytes += 2 * b * K + 2 * b * N if op == "adapters" else 0
        flops += 2 * b * (ranks * K + N * case["R"])
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------ the definitions, in 64 bits

def _exact_norm(s):
    t = s["x"].double()
    if s["res"] is not None:
        t += s["res"].double()
    t = t[:, :s["K"]]
    rms = torch.sqrt((t * t).sum(1) / s["K"] + EPS)
    v = t / rms[:, None] * s["weight"].double()[None, :]
    step = v.abs().max(1).values / 127
    codes = torch.clamp(torch.round(v / step[:, None]), -127, 127)
    return t, v, codes, step


def _exact_product(rows, s):
    ints = s["codes"].double()[:s["N"], :s["K"]].sub_(128)
    return torch.mm(rows, ints.t().contiguous()) * s["w_scale"]


def _exact_adapters(x, base, s):
    out = base.clone()
    for a in range(s["A"].shape[0]):
        rows = torch.nonzero(s["ids"] == a)[:, 0]
        if not rows.numel():
            continue
        first = 0
        for i, end in enumerate(s["ends"]):
            down = s["A"][a, i * s["R"]:(i + 1) * s["R"], :s["K"]].double()
            up = s["B"][a, first:end].double()
            inner = torch.mm(x[rows], down.t().contiguous())
            out[rows, first:end] += torch.mm(inner, up.t().contiguous()) * s["scale"][a].double()
            first = end
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "product":
        return {"y": _exact_product(s["q"].double()[:, :s["K"]] * s["q_scale"].double()[:, None], s)}
    if case["op"] == "adapters":
        return {"y": _exact_adapters(s["x"].double()[:, :s["K"]], s["base"].double(), s)}
    total, v, codes, step = _exact_norm(s)
    if case["op"] == "layer":
        return {"sum": total, "normed": v, "y": _exact_adapters(v, _exact_product(codes * step[:, None], s), s)}
    got = {}
    if s["res"] is not None:
        got["sum"] = total
    if s["fp16"]:
        got["y"] = v
    if s["int8"]:
        got["codes"] = codes * step[:, None]
        got["scale"] = step
    return got
