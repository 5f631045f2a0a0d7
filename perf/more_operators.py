"""The library's expert router and its microscaled 4-bit operators as they are
measured: cases, inputs, one pass through each operator, its work, and its
result in 64 bits.

Kinds of case
  route     the experts of each token from the router's logits (T x E) and
            their weights, and the gradient of the logits from that of the
            weights.  Scores are the row's softmax or each logit's sigmoid; a
            bias for balance, where there is one, is added to the scores for
            the choice alone; with groups, the choice is made among the experts
            of the `keep` groups whose two best (biased) scores sum highest.  The k
            chosen are in falling order, ties to the lowest number.  Weights
            are the chosen scores, divided by their sum where `renorm`, times
            `scale`.  A logit of minus infinity is an expert that cannot be
            chosen; a choice that no expert is left for is -1 and weighs 0.
  quant     rows of 16-bit values to microscaled 4-bit floating point: E2M1
            values in blocks of 32 along a row, each block with the power of
            two 2^(floor(log2(largest magnitude)) - 2) as its scale; rounding
            to nearest, ties to even, and what is above 6 scales becomes 6.
            With k > 0 the rows go to the k places of their token in a sort
            by expert; rows of dropped choices are zero.  The result is
            returned as the 16-bit values that it stands for.
  linear4   y = epi(x W^T): the activation rows are quantised as above, then
            multiplied by weights held in the same format (N x K).
  experts4  the experts' products on quantised rows sorted by expert and
            quantised weights (E x N x K): serving.

Where `own` is false `run` uses elementary torch operations in 32 bits (the
order of scores in 64: neighbours may differ by less than 32 bits hold) and
rounds once at the end; where it is true it calls the library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def listed():
    return [
        # routing of one step of a small decode batch, two of eight experts: launch latency
        dict(name="route_decode", kind="route", T=16, E=8, k=2, score="softmax", bias=False, groups=1, keep=1,
             renorm=True, scale=1.0, masked=0, dtype="bf16"),
        # a training batch over many experts, plain softmax weights, some padding tokens
        dict(name="route_train", kind="route", T=8192, E=128, k=8, score="softmax", bias=False, groups=1, keep=1,
             renorm=False, scale=1.0, masked=100, dtype="f32"),
        # a training batch with balanced sigmoid scores and groups of experts, odd number of tokens
        dict(name="route_groups", kind="route", T=16383, E=256, k=8, score="sigmoid", bias=True, groups=8, keep=4,
             renorm=True, scale=2.5, masked=0, dtype="f32"),
        # activations of a small decode batch
        dict(name="quant_decode", kind="quant", M=16, K=8192, k=0, E=1, drop=0, dtype="bf16"),
        # a whole prompt's activations
        dict(name="quant_prompt", kind="quant", M=16384, K=8192, k=0, E=1, drop=0, dtype="bf16"),
        # a batch's rows sorted by expert and quantised, a last block of 24, a few choices dropped
        dict(name="quant_sorted", kind="quant", M=8191, K=2040, k=6, E=64, drop=77, dtype="f16"),
        # one token of one sequence being decoded: weight streaming
        dict(name="linear4_decode_1", kind="linear4", M=1, N=8192, K=8192, dtype="bf16", relu=False),
        # a small decode batch through a wide layer
        dict(name="linear4_decode_16", kind="linear4", M=16, N=14336, K=4096, dtype="f16", relu=True),
        # a prompt batch whose sizes are no multiples of any tile, with ReLU
        dict(name="linear4_ragged", kind="linear4", M=3000, N=5000, K=4000, dtype="f16", relu=True),
        # a whole prompt through a large layer
        dict(name="linear4_prompt", kind="linear4", M=8192, N=8192, K=8192, dtype="bf16", relu=False),
        # a small decode batch: a few rows on some of the experts, weight streaming
        dict(name="experts4_decode", kind="experts4", R=32, E=16, K=4096, N=4096, tail=0, skew=1.0, dtype="bf16"),
        # a prompt batch on many experts, some choices dropped
        dict(name="experts4_prompt", kind="experts4", R=16384, E=64, K=4096, N=4096, tail=200, skew=0.5, dtype="f16"),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["route", "quant", "linear4", "experts4"])
    half = rng.choice(["bf16", "f16"])
    if kind == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * max(1, _log(rng, 2, 256) // groups)
        keep = rng.randint(1, groups)
        k = rng.randint(1, min(8, keep * (E // groups)))
        T = _log(rng, 1, 16383)
        return dict(kind=kind, T=T, E=E, k=k, score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5,
                    groups=groups, keep=keep, renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]),
                    masked=rng.choice([0, T // 50, T // 3]), dtype=rng.choice(["f32", "f32", "bf16", "f16"]))
    if kind == "quant":
        k = rng.choice([0, 0, 1, 2, 6, 8])
        M = _log(rng, 1, 16384 if k == 0 else 8191)
        K = _log(rng, 32, 8192)
        while M * K * max(1, k) > 16384 * 8192:        # no more than the largest listed case
            M //= 2
        E = max(k, _log(rng, 2, 256)) if k else 1
        return dict(kind=kind, M=M, K=K, k=k, E=E, drop=rng.choice([0, M * k // 50, M * k // 3]), dtype=half)
    if kind == "linear4":
        return dict(kind=kind, M=_log(rng, 1, 8192), N=_log(rng, 64, 8192), K=2 * _log(rng, 32, 4096), dtype=half,
                    relu=rng.random() < 0.5)
    E = _log(rng, 1, 64)
    K, N = 2 * _log(rng, 32, 2048), _log(rng, 64, 4096)
    R = _log(rng, 1, 16384)
    return dict(kind=kind, R=R, E=E, K=K, N=N, tail=rng.choice([0, R // 40, R // 5]),
                skew=rng.choice([0.0, 0.5, 2.0]), dtype=half)


# ------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _pitched(shape, dtype):
    """Storage for a row-major tensor whose row pitch is a multiple of 16
    bytes, as the library asks; a view of `shape`."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    pitch = -(-shape[-1] // per) * per
    return torch.zeros(*shape[:-1], pitch, dtype=dtype, device="cuda")[..., :shape[-1]]


def _activations(g, M, K, dtype):
    x = torch.randn((M, K), generator=g, device="cuda")
    x *= 1 + 9 * (torch.rand((1, K), generator=g, device="cuda") < 0.01)       # a few large channels
    out = _pitched((M, K), dtype)
    out.copy_(x)
    return out


def _quantised(g, shape, about):
    """Random codes of even K, with scales for values of about `about`."""
    K = shape[-1]
    codes = _pitched(shape[:-1] + (K // 2,), torch.uint8)
    scales = _pitched(shape[:-1] + (-(-K // 32),), torch.uint8)
    base = 127 + math.floor(math.log2(about / 2.5))
    for c, s in zip(codes, scales) if len(shape) == 3 else [(codes, scales)]:  # expert by expert: no large copies
        c.copy_(torch.randint(0, 256, c.shape, generator=g, device="cuda", dtype=torch.uint8))
        s.copy_(torch.randint(base - 1, base + 2, s.shape, generator=g, device="cuda", dtype=torch.uint8))
    return codes, scales


def _choices(g, T, k, E, drop):
    """T x k distinct expert numbers per token, some experts liked more, and
    `drop` of them replaced by numbers that name no expert."""
    liked = torch.randn((1, E), generator=g, device="cuda")
    ids = (torch.randn((T, E), generator=g, device="cuda") + liked).topk(k, dim=1).indices.to(torch.int32)
    if drop:
        gone = torch.randperm(T * k, generator=g, device="cuda")[:drop]
        ids.view(-1)[gone] = torch.where(gone % 2 == 0, -1, E).to(torch.int32)
    return ids.contiguous()


def _groups(case, g):
    """Row counts of the experts (a host list) and the offsets of their groups."""
    R, E = case["R"] - case["tail"], case["E"]
    share = torch.softmax(torch.randn((E,), generator=g, device="cuda") * case["skew"], 0)
    counts = torch.floor(share * R).to(torch.int64)
    counts[int(share.argmax())] += R - int(counts.sum())
    offsets = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offsets[1:] = counts.cumsum(0)
    return counts.tolist(), offsets


def _inputs(case, seed):
    g = _gen(seed)
    dt = DTYPES[case["dtype"]]
    kind = case["kind"]
    s = dict(case=case)
    if kind == "route":
        T, E = case["T"], case["E"]
        x = torch.randn((T, E), generator=g, device="cuda") * 1.5
        if case["masked"]:                             # padding tokens: no expert for them
            x[torch.randperm(T, generator=g, device="cuda")[:case["masked"]]] = -math.inf
        s["logits"] = x.to(dt)
        s["bias"] = torch.randn((E,), generator=g, device="cuda") * 0.05 if case["bias"] else None
        s["dw"] = torch.randn((T, case["k"]), generator=g, device="cuda")
    elif kind == "quant":
        s["x"] = _activations(g, case["M"], case["K"], dt)
        if case["k"]:
            s["ids"] = _choices(g, case["M"], case["k"], case["E"], case["drop"])
    elif kind == "linear4":
        s["x"] = _activations(g, case["M"], case["K"], dt)
        s["w"], s["ws"] = _quantised(g, (case["N"], case["K"]), 1 / math.sqrt(case["K"]))
    else:
        s["counts"], s["offsets"] = _groups(case, g)
        s["x"], s["xs"] = _quantised(g, (case["R"], case["K"]), 1.0)
        s["w"], s["ws"] = _quantised(g, (case["E"], case["N"], case["K"]), 1 / math.sqrt(case["K"]))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if case["kind"] == "route" and own:
        s["logits"].requires_grad_(True)
    if case["kind"] == "quant" and case["k"]:          # the sort that came before
        if own:
            import tiled_dense_gemm_tma_b200 as tg
            s["plan"] = tg.expert_sort(s["ids"], case["E"])
        else:
            s["kept"], s["pos"] = _plain_sort(s["ids"], case["E"])
    return s


# -------------------------------------------------------------- plain forms

_TABLE = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _plain_sort(ids, E):
    flat = ids.reshape(-1).to(torch.int64)
    kept = (flat >= 0) & (flat < E)
    src = torch.argsort(torch.where(kept, flat, E), stable=True)
    pos = torch.empty_like(src)
    pos[src] = torch.arange(src.numel(), device=src.device)
    return kept.view(ids.shape), pos.view(ids.shape)


def _power(e):
    """2^e in 32 bits, -126 <= e <= 127, from its bits: a power function may miss it by a bit."""
    return ((e + 127) << 23).view(torch.float32)


def _plain_decode(codes, scales, K):
    """The 32-bit values of a matrix of codes and its blocks' scales."""
    table = torch.tensor(_TABLE + tuple(-v for v in _TABLE), device=codes.device)
    rows = codes.shape[0]
    v = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), 2).reshape(rows, -1)
    return (v * _power(scales.int() - 127).repeat_interleave(32, 1)[:, :v.shape[1]])[:, :K]


def _plain_quant(x):
    """The 32-bit values that x becomes."""
    M, K = x.shape
    f = torch.zeros(M, -(-K // 32) * 32, device=x.device)
    f[:, :K] = x.float()
    b = f.view(M, -1, 32)
    top = b.abs().amax(2, keepdim=True)
    e = (torch.frexp(top).exponent - 3).clamp(-126, 126)   # frexp's mantissa is below 1
    y = b.abs() * _power(-e)
    i = ((y > 0.25).long() + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0))
    v = torch.tensor(_TABLE, device=x.device)[i] * _power(e)
    return torch.where(b < 0, -v, v).view(M, -1)[:, :K]


def _plain_route(s):
    case = s["case"]
    T, E, k, groups = case["T"], case["E"], case["k"], case["groups"]
    x = s["logits"].double()
    live = x > -math.inf
    top = torch.where(live.any(1, keepdim=True), x.amax(1, keepdim=True), 0.0)
    if case["score"] == "softmax":
        e = torch.exp(x - top)
        p = e / e.sum(1, keepdim=True).clamp(min=1.0)
    else:
        p = 1 / (1 + torch.exp(-x))
    key = x if s["bias"] is None else p + s["bias"].double()
    key = torch.where(live, key, -math.inf)
    if groups > 1:
        both = p if s["bias"] is None else p + s["bias"].double()
        both = torch.where(live, both, -math.inf).view(T, groups, -1).sort(2, descending=True).values
        best = both[:, :, 0]
        if both.shape[2] > 1:
            best = best + torch.where(both[:, :, 1] > -math.inf, both[:, :, 1], 0.0)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :case["keep"]]
        keep = torch.zeros(T, groups, dtype=torch.bool, device=x.device)
        keep.scatter_(1, order, True)
        key = torch.where(keep.repeat_interleave(E // groups, 1), key, -math.inf)
    val, ids = torch.sort(key, dim=1, descending=True, stable=True)
    val, ids = val[:, :k], ids[:, :k]
    has = val > -math.inf
    p = p.float()
    w = torch.where(has, p.gather(1, ids), 0.0)
    dw = torch.where(has, s["dw"], 0.0) * case["scale"]
    if case["renorm"]:
        total = w.sum(1, keepdim=True)
        total = torch.where(total > 0, total, 1.0)
        w = w / total
        dw = (dw - (dw * w).sum(1, keepdim=True)) / total
    ds = torch.zeros(T, E, device=x.device).scatter_add_(1, ids, torch.where(has, dw, 0.0))
    if case["score"] == "softmax":
        dx = p * (ds - (ds * p).sum(1, keepdim=True))
    else:
        dx = ds * p * (1 - p)
    return [torch.where(has, ids, -1).to(torch.int32), w * case["scale"], dx.to(s["logits"].dtype)]


def _plain_sorted_quant(s):
    case = s["case"]
    v = _plain_quant(s["x"]).to(s["x"].dtype)
    if not case["k"]:
        return v
    out = torch.zeros(case["M"] * case["k"], case["K"], dtype=v.dtype, device=v.device)
    for j in range(case["k"]):
        out[s["pos"][:, j]] = torch.where(s["kept"][:, j, None], v, 0)
    return out


def _plain_linear4(s):
    case = s["case"]
    y = _plain_quant(s["x"]) @ _plain_decode(s["w"], s["ws"], case["K"]).t()
    if case["relu"]:
        y = torch.where(y > 0, y, torch.zeros_like(y))
    return y.to(s["x"].dtype)


def _plain_experts4(s):
    case = s["case"]
    y = torch.zeros(case["R"], case["N"], dtype=DTYPES[case["dtype"]], device=s["x"].device)
    a = 0
    for e, n in enumerate(s["counts"]):
        if n:
            xe = _plain_decode(s["x"][a:a + n], s["xs"][a:a + n], case["K"])
            y[a:a + n] = (xe @ _plain_decode(s["w"][e], s["ws"][e], case["K"]).t()).to(y.dtype)
        a += n
    return y


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    kind = case["kind"]
    if not own:
        return {"route": _plain_route, "quant": _plain_sorted_quant, "linear4": _plain_linear4,
                "experts4": _plain_experts4}[kind](s)
    import tiled_dense_gemm_tma_b200 as tg
    if kind == "route":
        ids, w = tg.expert_route(s["logits"], case["k"], bias=s["bias"], score=case["score"], groups=case["groups"],
                                 topk_groups=case["keep"], renorm=case["renorm"], scale=case["scale"])
        dx, = torch.autograd.grad(w, s["logits"], s["dw"])
        return [ids, w.detach(), dx]
    if kind == "quant":
        q, qs = tg.quant_mxfp4(s["x"], plan=s.get("plan"))
        return tg.dequant_mxfp4(q, qs, case["K"], out_dtype=s["x"].dtype)
    if kind == "linear4":
        q, qs = tg.quant_mxfp4(s["x"])
        return tg.gemm_mxfp4(q, qs, s["w"], s["ws"], out_dtype=s["x"].dtype, relu=case["relu"])
    return tg.gemm_grouped_mxfp4(s["x"], s["xs"], s["offsets"], s["w"], s["ws"], out_dtype=DTYPES[case["dtype"]])


def _held(rows, K):
    """Bytes of a matrix in 4-bit blocks."""
    return rows * (-(-K // 2) + -(-K // 32))


def work(case):
    kind = case["kind"]
    if kind == "route":
        T, E, k = case["T"], case["E"], case["k"]
        wide = 4 if case["dtype"] == "f32" else 2
        # logits read, their gradient written; numbers and weights out, the weights' gradient in
        return dict(bytes=2 * wide * T * E + 12 * T * k + (4 * E if case["bias"] else 0), flops=8 * T * E)
    if kind == "quant":
        M, K, k = case["M"], case["K"], case["k"]
        n = M * max(1, k)
        # rows read, codes and scales written; those read, values written
        return dict(bytes=2 * M * K + 2 * _held(n, K) + 2 * n * K + 4 * M * k, flops=3 * M * K + n * K)
    if kind == "linear4":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=2 * M * K + _held(N, K) + 2 * M * N, flops=2 * M * N * K + 3 * M * K)
    R, E, K, N = case["R"], case["E"], case["K"], case["N"]
    live = R - case["tail"]
    # fewer rows than experts touch fewer weights
    busy = min(E, live)
    return dict(bytes=_held(live, K) + busy * _held(N, K) + 2 * R * N + 4 * (E + 1), flops=2 * live * K * N)


# ------------------------------------------------------- 64-bit definitions

def _exact_quant(x):
    """Rows in 64 bits, block by block: the nearest multiple of the spacing
    that E2M1 has at each magnitude."""
    M, K = x.shape
    out = torch.zeros(M, K, dtype=torch.float64, device=x.device)
    step = max(32, (1 << 24) // max(1, K) // 32 * 32)
    for a in range(0, M, step):
        part = torch.nn.functional.pad(x[a:a + step].double(), (0, -K % 32)).unflatten(1, (-1, 32))
        top = torch.linalg.vector_norm(part, math.inf, dim=2, keepdim=True)
        # the power of two at or below the largest magnitude is its bits without the mantissa
        scale = torch.where(top > 0, (top.view(torch.int64) >> 52 << 52).view(torch.float64) / 4, 1.0)
        y = part / scale
        space = torch.where(y.abs() < 2, 0.5, torch.where(y.abs() < 4, 1.0, 2.0))
        y = ((y / space).round() * space).clamp(-6, 6) * scale
        out[a:a + step] = y.flatten(1)[:, :K]
    return out


def _exact_held(codes, scales, K):
    """Codes and scales in 64 bits, from the bits of each code: sign,
    exponent with bias 1, mantissa."""
    c = torch.stack((codes.bitwise_and(15), codes.bitwise_right_shift(4)), -1).flatten(-2).to(torch.int64)
    ex, man = (c >> 1) & 3, (c & 1).double()
    v = torch.where(ex == 0, man / 2, (1 + man / 2) * (1 << (ex - 1).clamp(min=0)).double())
    v = torch.where(c >= 8, -v, v)
    block = torch.div(torch.arange(v.shape[-1], device=v.device), 32, rounding_mode="floor")
    up = ((scales.to(torch.int64) - 127 + 1023) << 52).view(torch.float64)
    return (v * up.index_select(-1, block))[..., :K]


def _exact_route(case, s):
    T, E, k = case["T"], case["E"], case["k"]
    x = s["logits"].double().requires_grad_(True)
    out = torch.isneginf(x.detach())
    gone = out.all(1)
    safe = torch.where(gone[:, None], 0.0, x)
    p = torch.softmax(safe, 1) if case["score"] == "softmax" else torch.sigmoid(safe)
    score = p.detach() if s["bias"] is None else p.detach() + s["bias"].double()
    rank = x.detach() if s["bias"] is None else score
    number = torch.arange(E, device=x.device).expand(T, E)
    allowed = ~out
    if case["groups"] > 1:
        per = E // case["groups"]
        parts = score.masked_fill(out, -math.inf).unflatten(1, (-1, per))
        best = parts.topk(min(2, per), 2).values
        best[:, :, 1:] = best[:, :, 1:].masked_fill(torch.isneginf(best[:, :, 1:]), 0.0)
        best = best.sum(2)
        inside = torch.zeros_like(allowed)
        which = torch.arange(case["groups"], device=x.device).expand(T, -1)
        left = torch.ones_like(best, dtype=torch.bool)
        for _ in range(case["keep"]):
            high = best.masked_fill(~left, -math.inf).amax(1, keepdim=True)
            first = which.masked_fill(~(left & (best == high)), case["groups"]).amin(1, keepdim=True)
            left &= which != first
            inside |= torch.div(number, per, rounding_mode="floor") == first
        allowed = allowed & inside
    ids = torch.full((T, k), -1, dtype=torch.int64, device=x.device)
    for j in range(k):
        high = rank.masked_fill(~allowed, -math.inf).amax(1, keepdim=True)
        first = number.masked_fill(~(allowed & (rank == high)), E).amin(1, keepdim=True)
        ids[:, j] = torch.where(first[:, 0] < E, first[:, 0], -1)
        allowed = allowed & (number != first)
    has = ids >= 0
    w = torch.where(has, p.gather(1, ids.clamp(min=0)), 0.0)
    if case["renorm"]:
        w = w / torch.where(has.any(1), w.sum(1), 1.0)[:, None]
    w = w * case["scale"]
    dx, = torch.autograd.grad(w, x, s["dw"].double())
    return [ids.to(torch.int32), w.detach(), dx]


def exact(case, seed):
    """What run returns, from the definitions, in 64 bits."""
    s = _inputs(case, seed)
    kind = case["kind"]
    if kind == "route":
        return _exact_route(case, s)
    if kind == "quant":
        v = _exact_quant(s["x"])
        if not case["k"]:
            return v
        M, k, E = case["M"], case["k"], case["E"]
        buckets = [[] for _ in range(E + 1)]
        for i, e in enumerate(s["ids"].reshape(-1).tolist()):
            buckets[e if 0 <= e < E else E].append(i)
        kept = sum(len(b) for b in buckets[:E])
        src = torch.tensor([i for b in buckets for i in b], dtype=torch.int64, device="cuda")
        out = v.index_select(0, torch.div(src, k, rounding_mode="floor"))
        out[kept:] = 0
        return out
    if kind == "linear4":
        y = torch.einsum("mk,nk->mn", _exact_quant(s["x"]), _exact_held(s["w"], s["ws"], case["K"]))
        return y.clamp(min=0) if case["relu"] else y
    cut = s["offsets"].tolist()
    y = torch.zeros(case["R"], case["N"], dtype=torch.float64, device="cuda")
    for e in range(case["E"]):
        part = slice(cut[e], cut[e + 1])
        y[part] = torch.einsum("rk,nk->rn", _exact_held(s["x"][part], s["xs"][part], case["K"]),
                               _exact_held(s["w"][e], s["ws"][e], case["K"]))
    return y
