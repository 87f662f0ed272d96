"""Timed cases of the operators around the quantized projection.

The library multiplies activations by quantized weights.  These are the operators that a
serving step runs next to that product:

  lora     low-rank adapters of many requests, added to the projection's output
  norm     residual addition and root-mean-square norm, which makes the projection's input
           (in 8 bits: the packed layout of 64-column groups with fp16 scale and zero)
  beam     beam search's selection over beams and vocabulary, after the LM head
  reorder  the beams' states (caches, token histories) moved to their new places

`run` computes them in plain torch operations, or, where `own` is set, by the library's
entry points.  Sizes are those of the workloads in `workloads/` or generic.
"""
import math

import torch

own = False

_DTYPE = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2, "q8": 1}
EPS = 1e-6


def listed():
    return [
        # q/k/v of a 896-wide layer for one request with one adapter: latency
        {"name": "lora one token", "op": "lora", "rows": 1, "segments": 1, "K": 896, "Ns": "896,128,128",
         "R": 16, "adapters": 4, "x": "f32", "w": "f16", "mixed": False},
        # one decode step of 64 requests over 48 adapters of mixed ranks, q/k/v of a 4096-wide layer
        {"name": "lora decode 64", "op": "lora", "rows": 64, "segments": 64, "K": 4096, "Ns": "4096,1024,1024",
         "R": 32, "adapters": 48, "x": "f32", "w": "bf16", "mixed": True},
        # seven prompts of different lengths through gate/up of a 4096-wide layer
        {"name": "lora prompts", "op": "lora", "rows": 4100, "segments": 7, "K": 4096, "Ns": "12288,12288",
         "R": 16, "adapters": 8, "x": "bf16", "w": "bf16", "mixed": False},
        # a few short prompts through a down projection, adapters of rank 128
        {"name": "lora rank 128", "op": "lora", "rows": 777, "segments": 5, "K": 4864, "Ns": "896",
         "R": 128, "adapters": 5, "x": "bf16", "w": "f16", "mixed": True},
        # the norm before one token's projections: latency
        {"name": "norm one token", "op": "norm", "rows": 1, "D": 896, "x": "f32", "res": "f32", "w": "f16", "out": "f32"},
        # per-head norm of 2048 tokens of 16 heads
        {"name": "norm heads", "op": "norm", "rows": 32768, "D": 128, "x": "bf16", "res": "", "w": "bf16", "out": "bf16"},
        # a prompt's rows between two layers: fp32 projection output, bf16 residual and bf16 projection input
        {"name": "norm prompt", "op": "norm", "rows": 8192, "D": 4096, "x": "f32", "res": "bf16", "w": "bf16", "out": "bf16"},
        # the same with rows kept in 8 bits
        {"name": "norm 8 bits", "op": "norm", "rows": 2048, "D": 4096, "x": "f32", "res": "f32", "w": "f16", "out": "q8"},
        # one request of four beams, an odd vocabulary
        {"name": "beam one request", "op": "beam", "batch": 1, "beams": 4, "V": 32003, "n_out": 4, "finished": False, "first": False},
        # 32 requests of eight beams over a large vocabulary, twice as many candidates as beams
        {"name": "beam batch", "op": "beam", "batch": 32, "beams": 8, "V": 151936, "n_out": 16, "finished": True, "first": False},
        # the token history of one request: latency
        {"name": "reorder tokens", "op": "reorder", "batch": 1, "beams": 4, "states": 1, "parts": 1, "bytes": 132, "room": 8192},
        # keys and values of eight layers, 8 heads of 128 in 16 bits, 1000 of 1024 places in use
        {"name": "reorder caches", "op": "reorder", "batch": 8, "beams": 4, "states": 16, "parts": 8, "bytes": 256000, "room": 262144},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _draw_lora(rng):
    rows = _spread(rng, 1, 4100)
    segments = rows if rows <= 256 and rng.random() < 0.5 else min(rows, _spread(rng, 1, 40))
    ns = [_spread(rng, 100, 12288) for _ in range(rng.randint(1, 3))]
    return {"op": "lora", "rows": rows, "segments": segments, "K": 64 * _spread(rng, 2, 192),
            "Ns": ",".join(map(str, ns)), "R": rng.choice([8, 16, 24, 32, 64, 128]),
            "adapters": _spread(rng, 1, 64), "x": rng.choice(["f32", "bf16"]), "w": rng.choice(["f16", "bf16"]),
            "mixed": rng.random() < 0.5}


def _draw_norm(rng):
    out = rng.choice(["f32", "bf16", "f16", "q8"])
    D = 64 * _spread(rng, 1, 256) if out == "q8" or rng.random() < 0.5 else _spread(rng, 33, 16384)
    return {"op": "norm", "rows": _spread(rng, 1, 32768), "D": D, "x": rng.choice(["f32", "bf16", "f16"]),
            "res": rng.choice(["", "f32", "bf16", "f16"]), "w": rng.choice(["f32", "bf16", "f16"]), "out": out}


def _draw_beam(rng):
    beams = rng.choice([1, 2, 3, 4, 5, 8, 16, 32])
    return {"op": "beam", "batch": _spread(rng, 1, 64), "beams": beams, "V": _spread(rng, 1000, 151936),
            "n_out": min(64, beams * rng.randint(1, 2)), "finished": rng.random() < 0.5, "first": rng.random() < 0.2}


def _draw_reorder(rng):
    step = rng.choice([1, 4, 16, 256])
    room = step * max(1, _spread(rng, 128, 262144) // step)
    return {"op": "reorder", "batch": _spread(rng, 1, 32), "beams": rng.choice([2, 3, 4, 5, 8, 16, 32]),
            "states": _spread(rng, 1, 48), "parts": _spread(rng, 1, 16),
            "bytes": step * max(1, int(room * rng.uniform(0.1, 1.0)) // step), "room": room}


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 200)


def draw(rng):
    pick = rng.choice([_draw_lora, _draw_norm, _draw_beam, _draw_reorder])
    most = max(_cost(c) for c in listed() if c["op"] == pick.__name__[6:])
    while True:
        case = pick(rng)
        if case["op"] == "reorder":
            size = case["batch"] * case["beams"] * case["states"] * case["parts"] * case["room"]
            if size > 1.5e9:
                continue
        if _cost(case) <= most:
            return case


def _ints(text):
    return [int(t) for t in text.split(",")]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 7919 + 17)
    return g


def _normal(g, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def prepare(case, seed):
    return {"lora": _prepare_lora, "norm": _prepare_norm, "beam": _prepare_beam,
            "reorder": _prepare_reorder}[case["op"]](case, _gen(seed))


def _prepare_lora(case, g):
    rows, S, K, R, n = (case[k] for k in ("rows", "segments", "K", "R", "adapters"))
    x = _normal(g, (rows, K), _DTYPE[case["x"]])
    if S == rows:
        start = torch.arange(rows + 1, dtype=torch.int32, device="cuda")
    else:                                           # cuts at random places: ragged, some empty
        cuts = torch.randint(0, rows + 1, (S - 1,), generator=g, device="cuda").sort().values
        ends = torch.tensor([0, rows], device="cuda")
        start = torch.cat([ends[:1], cuts, ends[1:]]).to(torch.int32)
    # -1: a request without an adapter
    adapter = torch.randint(-1 if S > 4 else 0, n, (S,), generator=g, device="cuda", dtype=torch.int32)
    choice = torch.tensor([max(1, R // 4), max(1, R // 2 - 1), R], dtype=torch.int32, device="cuda")
    ranks = choice[torch.randint(0, 3, (n,), generator=g, device="cuda")] if case["mixed"] else None
    scaling = 0.25 + torch.rand((n,), generator=g, device="cuda")
    w = _DTYPE[case["w"]]
    mats = []
    for N in _ints(case["Ns"]):
        mats.append((_normal(g, (n, R, K), w, 1 / math.sqrt(K)), _normal(g, (n, N, R), w, 1 / math.sqrt(R)),
                     _normal(g, (rows, N), torch.float32)))
    host = {"start": start.tolist(), "adapter": adapter.tolist(), "ranks": ranks.tolist() if case["mixed"] else [R] * n}
    return {"case": case, "x": x, "start": start, "adapter": adapter, "ranks": ranks, "scaling": scaling, "mats": mats,
            "host": host}


def _prepare_norm(case, g):
    rows, D = case["rows"], case["D"]
    x = _normal(g, (rows, D), _DTYPE[case["x"]])
    res = _normal(g, (rows, D), _DTYPE[case["res"]], 4.0) if case["res"] else None
    w = (1.0 + 0.2 * torch.randn((D,), generator=g, device="cuda")).to(_DTYPE[case["w"]])
    return {"case": case, "x": x, "res": res, "w": w}


def _prepare_beam(case, g):
    batch, beams, V = case["batch"], case["beams"], case["V"]
    logits = _normal(g, (batch * beams, V), torch.float32, 2.5)
    scores = (-20.0 * torch.rand((batch, beams), generator=g, device="cuda")).sort(dim=1, descending=True).values
    if case["first"]:                               # a search's first step: only beam 0 is alive
        scores[:, 1:] = -math.inf
    finished = (torch.rand((batch, beams), generator=g, device="cuda") < 0.2).to(torch.uint8) if case["finished"] else None
    return {"case": case, "logits": logits, "scores": scores, "finished": finished, "eos": V // 3, "pad": V // 2}


def _prepare_reorder(case, g):
    batch, beams, parts, room, used = (case[k] for k in ("batch", "beams", "parts", "room", "bytes"))
    states = [torch.randint(0, 256, (batch * beams, parts, room), generator=g, device="cuda", dtype=torch.uint8)
              for _ in range(case["states"])]
    parent = torch.randint(0, beams, (batch, beams), generator=g, device="cuda", dtype=torch.int32)
    return {"case": case, "states": states, "parent": parent, "used": used}


def run(state):
    return {"lora": _run_lora, "norm": _run_norm, "beam": _run_beam, "reorder": _run_reorder}[state["case"]["op"]](state)


def _run_lora(s):
    x, start, adapter, ranks, scaling = s["x"], s["start"], s["adapter"], s["ranks"], s["scaling"]
    ys = [m[2] for m in s["mats"]]
    if own:
        import quantized_matmul_02_b200 as qmm
        qmm.lora_add_batched(qmm.make_lora_descs([(x, A, B, y) for A, B, y in s["mats"]]), start, adapter,
                             ranks=ranks, scaling=scaling)
        return ys
    R = s["mats"][0][0].shape[1]
    if x.shape[0] == start.numel() - 1:             # one row a request: the requests' adapters, gathered
        live = (adapter >= 0).float()
        at = adapter.clamp(min=0).long()
        c = (live * scaling[at])[:, None]
        if ranks is not None:
            c = c * (torch.arange(R, device=x.device) < ranks[at][:, None]).float()
        for A, B, y in s["mats"]:
            v = torch.matmul(A[at].float(), x.float()[:, :, None])[:, :, 0] * c
            y += torch.matmul(B[at].float(), v[:, :, None])[:, :, 0]
        return ys
    # prompts: one product a request, as its rows lie together and its length is known on the host
    first, rank = s["host"]["start"], s["host"]["ranks"]
    for A, B, y in s["mats"]:
        for i, a in enumerate(s["host"]["adapter"]):
            if a < 0 or first[i] == first[i + 1]:
                continue
            r = rank[a]
            v = torch.matmul(x[first[i]:first[i + 1]].float(), A[a, :r].float().T) * scaling[a]
            y[first[i]:first[i + 1]] += torch.matmul(v, B[a, :, :r].float().T)
    return ys


def _run_norm(s):
    case, x, res, w = s["case"], s["x"], s["res"], s["w"]
    if own:
        import quantized_matmul_02_b200 as qmm
        if case["out"] != "q8":
            out = qmm.add_rmsnorm(x, w, EPS, residual=res, out_dtype=_DTYPE[case["out"]])
        else:
            codes, scale, zero = qmm.add_rmsnorm_q8(x, w, EPS, residual=res)
            out = ((codes.view(*scale.shape, 64) - zero[..., None]) * scale[..., None]).view(x.shape)
        return [out] if res is None else [out, res]
    h = x.float()
    if res is not None:
        h = h + res.float()
        res.copy_(h)
    v = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + EPS) * w.float()
    if case["out"] != "q8":
        out = v.to(_DTYPE[case["out"]])
    else:
        v = v.view(x.shape[0], -1, 64)
        lo, hi = v.amin(dim=2, keepdim=True).clamp(max=0), v.amax(dim=2, keepdim=True).clamp(min=0)
        scale = ((hi - lo) / 255).to(torch.float16).float().clamp(min=2.0 ** -24)
        zero = torch.round(-lo / scale)
        q = (torch.round(v / scale) + zero).clamp(0, 255)
        out = ((q - zero) * scale).to(torch.float16).view(x.shape)
    return [out] if res is None else [out, res]


def _run_beam(s):
    case, logits, scores, finished = s["case"], s["logits"], s["scores"], s["finished"]
    batch, beams, V, n = case["batch"], case["beams"], case["V"], case["n_out"]
    if own:
        import quantized_matmul_02_b200 as qmm
        return qmm.beam_select(logits, scores, n, finished=finished, eos=s["eos"], pad=s["pad"])
    # the best n of each beam, then the best n of all beams'; 64 bits where values next to each other are ordered
    value, token = torch.topk(logits, n, dim=1)
    token, order = token.sort(dim=1)                # equal totals: the lowest token first
    logp = value.gather(1, order).double() - torch.logsumexp(logits.double(), dim=1, keepdim=True)
    low = torch.arange(n, device=logits.device).expand_as(token)
    alive = scores.view(-1, 1) > -math.inf
    total = torch.where(alive, scores.double().view(-1, 1) + logp, -math.inf)
    token = torch.where(alive, token, low)
    done = torch.zeros_like(scores, dtype=torch.bool) if finished is None else finished.bool()
    if finished is not None:                        # a finished beam goes on through one pad token
        over = done.view(-1, 1)
        kept = torch.where(low == n - 1, s["pad"], low)
        total = torch.where(over, torch.where(low == n - 1, scores.double().view(-1, 1), -math.inf), total)
        token = torch.where(over, kept, token)
    best, at = torch.sort(total.view(batch, beams * n), dim=1, descending=True, stable=True)
    best, at = best[:, :n], at[:, :n]
    parent = at // n
    token = token.view(batch, beams * n).gather(1, at)
    ended = done.gather(1, parent) | (token == s["eos"])
    return best.float(), parent.int(), token.int(), ended.to(torch.uint8)


def _run_reorder(s):
    case, parent, used = s["case"], s["parent"], s["used"]
    batch, beams = case["batch"], case["beams"]
    if own:
        import quantized_matmul_02_b200 as qmm
        qmm.beam_reorder([t[:, :, :used] for t in s["states"]], parent)
        return s["states"]
    at = (parent.long() + beams * torch.arange(batch, device=parent.device)[:, None]).view(-1)
    for t in s["states"]:
        t[:, :, :used] = t[at, :, :used]
    return s["states"]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "lora":
        return _exact_lora(case, s)
    if case["op"] == "norm":
        return _exact_norm(case, s)
    return _exact_beam(case, s) if case["op"] == "beam" else None


def _exact_lora(case, s):
    """Row by row of the definition, all rows of one adapter at a time."""
    rows, R = case["rows"], case["R"]
    owner = torch.full((rows,), -1, dtype=torch.int64, device="cuda")
    edges = s["start"].cpu().numpy()
    for i, a in enumerate(s["adapter"].cpu().numpy()):
        owner[int(edges[i]):int(edges[i + 1])] = int(a)
    xd, out = s["x"].to(torch.float64), []
    for A, B, y in s["mats"]:
        yd = y.to(torch.float64)
        for a in range(case["adapters"]):
            mine = torch.nonzero(owner == a)[:, 0]
            if mine.numel() == 0:
                continue
            keep = int(s["ranks"][a]) if s["ranks"] is not None else R
            low = torch.einsum("mk,rk->mr", xd[mine], A[a, :keep].to(torch.float64))
            yd[mine] += s["scaling"][a].to(torch.float64) * torch.einsum("mr,nr->mn", low, B[a, :, :keep].to(torch.float64))
        out.append(yd)
    return out


def _exact_norm(case, s):
    h = s["x"].to(torch.float64)
    if s["res"] is not None:
        h += s["res"].to(torch.float64)
    power = torch.einsum("md,md->m", h, h) / case["D"]
    v = h / torch.sqrt(power + EPS)[:, None]
    v *= s["w"].to(torch.float64)
    if case["out"] == "q8":
        g = v.reshape(-1, 64)
        low = torch.minimum(g.min(1).values, torch.zeros((), dtype=torch.float64, device="cuda"))
        high = torch.maximum(g.max(1).values, torch.zeros((), dtype=torch.float64, device="cuda"))
        step = ((high - low) / 255).half().double()
        step[step < 2.0 ** -24] = 2.0 ** -24
        base = torch.round(low / -step)[:, None]
        code = torch.clamp(torch.round(g / step[:, None]) + base, 0, 255)
        v = ((code - base) * step[:, None]).reshape(v.shape)
    return [v] if s["res"] is None else [v, h]


def _exact_beam(case, s):
    """All beams x V totals of a request, in order."""
    batch, beams, V, n = case["batch"], case["beams"], case["V"], case["n_out"]
    scores, got = s["scores"].to(torch.float64), ([], [], [], [])
    for b in range(batch):
        total = torch.log_softmax(s["logits"][b * beams:(b + 1) * beams].to(torch.float64), 1)
        total += scores[b, :, None]
        over = s["finished"][b].bool() if s["finished"] is not None else torch.zeros(beams, dtype=torch.bool, device="cuda")
        total[over] = -math.inf
        total[over, s["pad"]] = scores[b, over]
        value, flat = torch.sort(total.reshape(-1), descending=True, stable=True)
        flat = flat[:n]
        got[0].append(value[:n])
        got[1].append(flat.div(V, rounding_mode="floor"))
        got[2].append(flat % V)
        got[3].append((over[got[1][-1]] | (got[2][-1] == s["eos"])).to(torch.uint8))
    value, parent, token, ended = (torch.stack(g) for g in got)
    return value, parent.to(torch.int32), token.to(torch.int32), ended


def work(case):
    """Bytes: each input read once, each output written once."""
    if case["op"] == "lora":
        rows, K, R = case["rows"], case["K"], case["R"]
        used = min(case["adapters"], case["segments"])
        Ns = _ints(case["Ns"])
        return {"bytes": rows * K * _BYTES[case["x"]] + sum(8 * rows * N + 2 * used * R * (K + N) for N in Ns),
                "flops": sum(2 * rows * R * (K + N) for N in Ns)}
    if case["op"] == "norm":
        each = _BYTES[case["x"]] + _BYTES[case["out"]] + (2 * _BYTES[case["res"]] if case["res"] else 0)
        return {"bytes": case["rows"] * case["D"] * each + case["D"] * _BYTES[case["w"]], "flops": 5 * case["rows"] * case["D"]}
    if case["op"] == "beam":
        n = case["batch"] * case["beams"] * case["V"]
        return {"bytes": 4 * n + 13 * case["batch"] * case["n_out"], "flops": 4 * n}
    # a beam whose parent is itself stays; the parents of the others are read once each
    W = case["beams"]
    one = case["batch"] * case["states"] * case["parts"] * case["bytes"]
    moved = W - 1
    read = W * (1 - (1 - 1 / W) ** W)
    return {"bytes": one * (moved + read), "flops": 0}
