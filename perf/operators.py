"""The library's 8-bit linear layer and mixture-of-experts operators as they
are measured: cases, inputs, one pass through each operator, its work, and
its result in 64 bits.

Kinds of case
  linear8   y = epi(x W): the activation rows are quantised to signed 8-bit
            integers with one scale per token, then multiplied by 8-bit
            weights with one scale per output channel.  x (M x K) and y
            (M x N) are 16-bit; W is stored K x N, or N x K (trans).
  route     tokens sorted by expert: from expert numbers (T x k) the sorted
            positions, the group offsets, the sorted rows, and the gradient
            of the tokens from the gradient of the sorted rows.  A number
            outside 0..E-1 is a dropped choice: it sorts behind the last
            group and its row is zero.
  combine   sorted rows back to tokens, weights applied, with the gradients
            of rows and weights.
  experts   the experts' products on sorted rows, forward and both
            gradients, 16-bit.
  experts8  the experts' products on 8-bit rows and weights (serving).

Where `own` is false `run` uses elementary torch operations in 32 bits and
rounds once at the end; where it is true it calls the library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def listed():
    return [
        # one token of one sequence being decoded: latency and weight streaming
        dict(name="linear8_decode_1", kind="linear8", M=1, N=8192, K=8192, dtype="bf16", trans=False, relu=False),
        # a small decode batch on weights stored out x in
        dict(name="linear8_decode_16", kind="linear8", M=16, N=8192, K=8192, dtype="f16", trans=True, relu=False),
        # a prompt batch whose sizes are no multiples of any tile, with ReLU
        dict(name="linear8_ragged", kind="linear8", M=3000, N=5000, K=4000, dtype="bf16", trans=False, relu=True),
        # a whole prompt through a large layer
        dict(name="linear8_prompt", kind="linear8", M=4096, N=8192, K=8192, dtype="bf16", trans=True, relu=False),
        # routing of a small decode batch: launch latency
        dict(name="route_decode", kind="route", T=16, k=2, E=8, H=4096, drop=0, dtype="bf16"),
        # routing of a training batch over many experts, a few choices dropped
        dict(name="route_train", kind="route", T=8192, k=8, E=128, H=2048, drop=100, dtype="bf16"),
        # results of a small decode batch joined again
        dict(name="combine_decode", kind="combine", T=16, k=2, E=8, H=4096, drop=0, dtype="bf16"),
        # a training batch joined again, odd row length, a few choices dropped
        dict(name="combine_train", kind="combine", T=8191, k=6, E=64, H=2040, drop=77, dtype="f16"),
        # a small training step: few rows per expert, odd sizes, empty experts
        dict(name="experts_small", kind="experts", R=777, E=16, K=1000, N=520, tail=5, skew=2.0, dtype="f16", trans=True),
        # a training step's worth of rows on large experts
        dict(name="experts_train", kind="experts", R=32768, E=32, K=4096, N=2048, tail=0, skew=0.5, dtype="bf16", trans=False),
        # a small decode batch: a few rows on some of the experts, weight streaming
        dict(name="experts8_decode", kind="experts8", R=32, E=16, K=4096, N=4096, tail=0, skew=1.0, dtype="bf16", trans=True),
        # a prompt batch on many experts
        dict(name="experts8_prompt", kind="experts8", R=16384, E=64, K=4096, N=4096, tail=0, skew=0.5, dtype="bf16", trans=False),
    ]


def _log(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["linear8", "route", "combine", "experts", "experts8"])
    dtype = rng.choice(["bf16", "f16"])
    if kind == "linear8":
        return dict(kind=kind, M=_log(rng, 1, 4096), N=_log(rng, 64, 8192), K=_log(rng, 64, 8192), dtype=dtype,
                    trans=rng.random() < 0.5, relu=rng.random() < 0.5)
    if kind in ("route", "combine"):
        E = _log(rng, 2, 256)
        T = _log(rng, 1, 8192)
        k = rng.randint(1, min(8, E))
        return dict(kind=kind, T=T, k=k, E=E, H=_log(rng, 64, 2048), drop=rng.choice([0, (T * k) // 50, (T * k) // 3]),
                    dtype=dtype)
    E = _log(rng, 1, 64)
    K, N = _log(rng, 64, 4096), _log(rng, 64, 4096)
    while E * K * N > 32 * 4096 * 2048:            # no more weights than the largest listed case
        E = max(1, E // 2)
    top = 32768 if kind == "experts" else 16384
    while top * K * N > 32768 * 4096 * 2048:       # nor more products
        top //= 2
    R = _log(rng, 1, top)
    return dict(kind=kind, R=R, E=E, K=K, N=N, tail=rng.choice([0, R // 40, R // 5]), skew=rng.choice([0.0, 0.5, 2.0]),
                dtype=dtype, trans=rng.random() < 0.5)


# ------------------------------------------------------------------- inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _pitched(shape, dtype):
    """Storage for a row-major tensor whose row pitch is a multiple of 16
    bytes, as the library asks; a view of `shape`."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    pitch = -(-shape[-1] // per) * per
    return torch.zeros(*shape[:-1], pitch, dtype=dtype, device="cuda")[..., :shape[-1]]


def _normal(g, shape, dtype, scale=1.0):
    out = _pitched(shape, dtype)
    if len(shape) == 3:                            # expert by expert: no large 32-bit copy
        for e in range(shape[0]):
            out[e] = torch.randn(shape[1:], generator=g, device="cuda") * scale
    else:
        out.copy_(torch.randn(shape, generator=g, device="cuda") * scale)
    return out


def _weights8(g, shape):
    out = _pitched(shape, torch.int8)
    for part in (out if len(shape) == 3 else [out]):
        part.copy_((torch.randn(part.shape, generator=g, device="cuda") * 32).round().clamp(-127, 127))
    return out


def _scales(g, shape, about):
    return (torch.rand(shape, generator=g, device="cuda") + 0.5) * about


def _choices(case, g):
    """T x k distinct expert numbers per token, some experts liked more, and
    `drop` of them replaced by numbers that name no expert."""
    T, k, E = case["T"], case["k"], case["E"]
    liked = torch.randn((1, E), generator=g, device="cuda")
    ids = (torch.randn((T, E), generator=g, device="cuda") + liked).topk(k, dim=1).indices.to(torch.int32)
    if case["drop"]:
        gone = torch.randperm(T * k, generator=g, device="cuda")[:case["drop"]]
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
    if kind == "linear8":
        M, N, K = case["M"], case["N"], case["K"]
        x = torch.randn((M, K), generator=g, device="cuda")
        x *= 1 + 9 * (torch.rand((1, K), generator=g, device="cuda") < 0.01)   # a few large channels
        s["x"] = _pitched((M, K), dt)
        s["x"].copy_(x)
        s["w"] = _weights8(g, (N, K) if case["trans"] else (K, N))
        s["ws"] = _scales(g, (N,), 1.0 / (32 * math.sqrt(K)))
    elif kind == "route":
        s["ids"] = _choices(case, g)
        s["x"] = _normal(g, (case["T"], case["H"]), dt)
        s["dxs"] = _normal(g, (case["T"] * case["k"], case["H"]), dt)
    elif kind == "combine":
        s["ids"] = _choices(case, g)
        s["ys"] = _normal(g, (case["T"] * case["k"], case["H"]), dt)
        s["wt"] = torch.softmax(torch.randn((case["T"], case["k"]), generator=g, device="cuda"), 1)
        s["dy"] = _normal(g, (case["T"], case["H"]), dt)
    else:
        R, E, K, N = case["R"], case["E"], case["K"], case["N"]
        s["counts"], s["offsets"] = _groups(case, g)
        shape = (E, N, K) if case["trans"] else (E, K, N)
        if kind == "experts":
            s["x"] = _normal(g, (R, K), dt)
            s["w"] = _normal(g, shape, dt, 1 / math.sqrt(K))
            s["dy"] = _normal(g, (R, N), dt)
        else:
            s["x"] = _weights8(g, (R, K))
            s["xs"] = _scales(g, (R,), 1.0 / 32)
            s["w"] = _weights8(g, shape)
            s["ws"] = _scales(g, (E, N), 1.0 / (32 * math.sqrt(K)))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    kind = case["kind"]
    if kind == "route":
        if own:
            s["x"].requires_grad_(True)
    elif kind == "combine":
        if own:                                     # the plan of the sort that came before
            import tiled_dense_gemm_tma_b200 as tg
            s["plan"] = tg.expert_sort(s["ids"], case["E"])
            s["ys"].requires_grad_(True)
            s["wt"].requires_grad_(True)
        else:
            s["kept"], s["pos"] = _plain_sort(s["ids"], case["E"])[2:]
    elif kind == "experts" and own:
        s["x"].requires_grad_(True)
        s["w"].requires_grad_(True)
    return s


# -------------------------------------------------------------- plain forms

def _plain_sort(ids, E):
    flat = ids.reshape(-1).to(torch.int64)
    kept = (flat >= 0) & (flat < E)
    group = torch.where(kept, flat, E)
    src = torch.argsort(group, stable=True)
    pos = torch.empty_like(src)
    pos[src] = torch.arange(src.numel(), device=src.device)
    counts = (group[:, None] == torch.arange(E, device=src.device)).sum(0)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=src.device)
    offsets[1:] = counts.cumsum(0)
    return offsets.to(torch.int32), src.to(torch.int32), kept.view(ids.shape), pos.view(ids.shape)


def _plain_linear8(s):
    case = s["case"]
    x = s["x"].float()
    top = x.abs().amax(1, keepdim=True)
    q = torch.where(top > 0, torch.round(x * 127 / top), torch.zeros_like(x))
    w = s["w"].float()
    y = q @ (w.t() if case["trans"] else w)
    y = y * (top / 127) * s["ws"]
    if case["relu"]:
        y = torch.where(y > 0, y, torch.zeros_like(y))
    return [y.to(s["x"].dtype), (top / 127)[:, 0]]


def _plain_route(s):
    case = s["case"]
    T, k, H = case["T"], case["k"], case["H"]
    offsets, src, kept, pos = _plain_sort(s["ids"], case["E"])
    live = (torch.arange(T * k, device=src.device) < offsets[-1])[:, None]
    xs = torch.where(live, s["x"][(src // k).long()], 0)
    dx = torch.zeros(T, H, device=src.device)
    for j in range(k):
        dx += torch.where(kept[:, j, None], s["dxs"][pos[:, j]].float(), 0)
    return [offsets, pos.to(torch.int32), src, xs, dx.to(s["x"].dtype)]


def _plain_combine(s):
    case = s["case"]
    T, k, H = case["T"], case["k"], case["H"]
    kept, pos = s["kept"], s["pos"]
    ys, wt, dy = s["ys"], s["wt"], s["dy"].float()
    y = torch.zeros(T, H, device=ys.device)
    dys = torch.zeros_like(ys)
    dwt = torch.zeros_like(wt)
    for j in range(k):
        row = torch.where(kept[:, j, None], ys[pos[:, j]].float(), 0)
        y += wt[:, j, None] * row
        dys[pos[:, j]] = torch.where(kept[:, j, None], wt[:, j, None] * dy, 0).to(ys.dtype)
        dwt[:, j] = (row * dy).sum(1)
    return [y.to(ys.dtype), dys, dwt]


def _plain_experts(s):
    case = s["case"]
    x, w, dy = s["x"], s["w"], s["dy"]
    y, dx, dw = torch.zeros_like(dy), torch.zeros_like(x), torch.zeros_like(w)
    a = 0
    for e, n in enumerate(s["counts"]):
        if n:
            xe, de, we = x[a:a + n].float(), dy[a:a + n].float(), w[e].float()
            if case["trans"]:
                y[a:a + n], dx[a:a + n], dw[e] = xe @ we.t(), de @ we, de.t() @ xe
            else:
                y[a:a + n], dx[a:a + n], dw[e] = xe @ we, de @ we.t(), xe.t() @ de
        a += n
    return [y, dx, dw]


def _plain_experts8(s):
    case = s["case"]
    y = torch.zeros(case["R"], case["N"], dtype=DTYPES[case["dtype"]], device=s["x"].device)
    a = 0
    for e, n in enumerate(s["counts"]):
        if n:
            we = s["w"][e].float()
            ye = s["x"][a:a + n].float() @ (we.t() if case["trans"] else we)
            y[a:a + n] = ye * s["xs"][a:a + n, None] * s["ws"][e]
        a += n
    return y


# ------------------------------------------------------------------ one pass

def run(s):
    case = s["case"]
    kind = case["kind"]
    if not own:
        return {"linear8": _plain_linear8, "route": _plain_route, "combine": _plain_combine,
                "experts": _plain_experts, "experts8": _plain_experts8}[kind](s)
    import tiled_dense_gemm_tma_b200 as tg
    if kind == "linear8":
        q, qs = tg.quant_i8(s["x"])
        y = tg.gemm_w8a8(q, qs, s["w"], s["ws"], out_dtype=s["x"].dtype, relu=case["relu"], trans_b=case["trans"])
        return [y, qs]
    if kind == "route":
        plan = tg.expert_sort(s["ids"], case["E"])
        xs = tg.expert_gather(s["x"], plan)
        dx, = torch.autograd.grad(xs, s["x"], s["dxs"])
        return [plan.offsets, plan.pos, plan.src, xs.detach(), dx]
    if kind == "combine":
        y = tg.expert_combine(s["ys"], s["plan"], s["wt"])
        dys, dwt = torch.autograd.grad(y, (s["ys"], s["wt"]), s["dy"])
        return [y.detach(), dys, dwt]
    if kind == "experts":
        w = s["w"].transpose(1, 2) if case["trans"] else s["w"]
        y = tg.expert_matmul(s["x"], w, s["offsets"])
        dx, dw = torch.autograd.grad(y, (s["x"], s["w"]), s["dy"])
        return [y.detach(), dx, dw]
    return tg.gemm_grouped_w8a8(s["x"], s["xs"], s["offsets"], s["w"], s["ws"], out_dtype=DTYPES[case["dtype"]],
                                trans_b=case["trans"])


def work(case):
    kind = case["kind"]
    if kind == "linear8":
        M, N, K = case["M"], case["N"], case["K"]
        return dict(bytes=2 * M * K + N * K + 4 * N + 2 * M * N + 4 * M, flops=2 * M * N * K + 3 * M * K)
    if kind == "route":
        T, k, H = case["T"], case["k"], case["H"]
        n = T * k
        # expert numbers in; offsets and both orders out; tokens read, sorted
        # rows written, then their gradient read and the tokens' written
        return dict(bytes=4 * n + 8 * n + 4 * (case["E"] + 1) + 2 * (2 * T * H + n * H + (n - case["drop"]) * H),
                    flops=n * H)
    if kind == "combine":
        T, k, H = case["T"], case["k"], case["H"]
        n = T * k
        # kept rows read (once, had the two passes been one), tokens written;
        # the tokens' gradient read, the rows' written; weights in, gradient out
        return dict(bytes=2 * ((n - case["drop"]) * H + 2 * T * H + n * H) + 12 * n, flops=5 * n * H)
    R, E, K, N = case["R"], case["E"], case["K"], case["N"]
    live = R - case["tail"]
    if kind == "experts":
        # x, w and dy read once; y, dx and dw written once
        return dict(bytes=2 * (live * (K + N) + R * (K + N) + 2 * E * K * N) + 4 * (E + 1), flops=6 * live * K * N)
    # fewer rows than experts touch fewer weights
    busy = min(E, live)
    return dict(bytes=live * (K + 4) + busy * (K * N + 4 * N) + 2 * R * N + 4 * (E + 1), flops=2 * live * K * N)


# ------------------------------------------------------- 64-bit definitions

def exact(case, seed):
    """What run returns, from the definitions, element by element in 64 bits."""
    s = _inputs(case, seed)
    kind = case["kind"]
    if kind == "linear8":
        x = s["x"].double()
        peak = torch.linalg.vector_norm(x, math.inf, dim=1)
        unit = peak / 127
        q = torch.zeros_like(x)
        some = peak > 0
        q[some] = (x[some] * 127.0 / peak[some][:, None]).round()
        w = s["w"].double()
        y = torch.einsum("mk,nk->mn" if case["trans"] else "mk,kn->mn", q, w)
        y = torch.einsum("mn,m,n->mn", y, unit, s["ws"].double())
        return [y.clamp(min=0) if case["relu"] else y, unit]
    if kind in ("route", "combine"):
        T, k, E, H = case["T"], case["k"], case["E"], case["H"]
        flat = s["ids"].reshape(-1).tolist()
        buckets = [[] for _ in range(E + 1)]
        for i, e in enumerate(flat):
            buckets[e if 0 <= e < E else E].append(i)
        order = [i for b in buckets for i in b]
        ends = [0]
        for b in buckets[:E]:
            ends.append(ends[-1] + len(b))
        src = torch.tensor(order, dtype=torch.int64, device="cuda")
        place = torch.zeros(T * k, dtype=torch.int64, device="cuda")
        place.scatter_(0, src, torch.arange(T * k, device="cuda"))
        n = ends[-1]
        token = torch.div(src[:n], k, rounding_mode="floor")
        if kind == "route":
            xs = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
            xs[:n] = s["x"].double().index_select(0, token)
            dx = torch.zeros(T, H, dtype=torch.float64, device="cuda").index_add_(0, token, s["dxs"][:n].double())
            return [torch.tensor(ends, dtype=torch.int32, device="cuda"), place.view(T, k).to(torch.int32),
                    src.to(torch.int32), xs, dx]
        each = s["wt"].double().reshape(-1)[src[:n]]
        rows = s["ys"][:n].double()
        back = s["dy"].double().index_select(0, token)
        y = torch.zeros(T, H, dtype=torch.float64, device="cuda").index_add_(0, token, rows * each[:, None])
        dys = torch.zeros(T * k, H, dtype=torch.float64, device="cuda")
        dys[:n] = back * each[:, None]
        dwt = torch.zeros(T * k, dtype=torch.float64, device="cuda")
        dwt[src[:n]] = torch.einsum("rh,rh->r", rows, back)
        return [y, dys, dwt.view(T, k)]
    R, E, K, N = case["R"], case["E"], case["K"], case["N"]
    cut = s["offsets"].tolist()
    y = torch.zeros(R, N, dtype=torch.float64, device="cuda")
    if kind == "experts8":
        for e in range(E):
            part = slice(cut[e], cut[e + 1])
            y[part] = torch.einsum("rk,nk->rn" if case["trans"] else "rk,kn->rn", s["x"][part].double(), s["w"][e].double())
            y[part] *= torch.outer(s["xs"][part].double(), s["ws"][e].double())
        return y
    dx = torch.zeros(R, K, dtype=torch.float64, device="cuda")
    dw = torch.zeros(tuple(s["w"].shape), dtype=torch.float64, device="cuda")
    io = "oi" if case["trans"] else "io"
    for e in range(E):
        part = slice(cut[e], cut[e + 1])
        xe, de, we = s["x"][part].double(), s["dy"][part].double(), s["w"][e].double()
        y[part] = torch.einsum("ri,%s->ro" % io, xe, we)
        dx[part] = torch.einsum("ro,%s->ri" % io, de, we)
        dw[e] = torch.einsum("ri,ro->%s" % io, xe, de)
    return [y, dx, dw]
