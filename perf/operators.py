"""What is measured of the two operators around the head loss: drawing tokens from
the head's logits, and the global gradient norm with clipping.

`run` computes them in plain torch operations, or (`own`) through the library's
public entry points.  A sampling case is rows x vocab logits with the requests'
settings and one given uniform number a row; a clipping case is a list of
gradient tensors, clipped into buffers of the same layout.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2}
LOG2E = 1.4426950408889634
UNIT = 2.0 ** 30  # the weight of a row's largest logit


def _sample(name, rows, vocab, dtype, settings, pitch=0, softcap=0.0, scale=1.0, masked=0.0):
    case = dict(op="sample", rows=rows, vocab=vocab, pitch=pitch or vocab, dtype=dtype,
                settings=settings, softcap=softcap, scale=scale, masked=masked)
    return dict(case, name=name) if name else case


def _clip(name, dtype, tensors, elements, spread=False, vectors=0, vector=0, over=4.0, scaled=1.0):
    case = dict(op="clip", dtype=dtype, tensors=tensors, elements=elements, spread=spread,
                vectors=vectors, vector=vector, over=over, scaled=scaled)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one interactive request: latency is all that counts
        _sample("one token", 1, 32000, "bf16", "chat"),
        # a small serving batch, every request with settings of its own (greedy ones too),
        # some of them with tokens forbidden by a grammar
        _sample("small batch", 16, 128256, "bf16", "mixed", masked=0.25),
        # fp32 logits with an odd vocabulary: rows off the 16-byte grid
        _sample("odd fp32 rows", 77, 32003, "fp32", "minp"),
        # a full serving batch; the head's columns are padded to its tile
        _sample("full batch", 256, 151936, "bf16", "mixed", pitch=152064),
        # a capped and scaled head in fp16
        _sample("capped head", 512, 128256, "fp16", "chat", softcap=30.0, scale=0.5),
        # policy rollouts: the model's own distribution, no filter
        _sample("rollout", 1024, 151936, "bf16", "own"),
        # rollouts drawn from the nucleus alone
        _sample("nucleus", 1024, 128256, "bf16", "nucleus"),
        # offline generation over very many short prompts
        _sample("offline", 8192, 32000, "bf16", "chat"),
        # a probe's weights and biases: a handful of small odd tensors
        _clip("small odd", "fp32", 14, 9001, spread=True),
        # adapters of every projection of a deep model: many small tensors
        _clip("adapters", "bf16", 448, 65536),
        # the head's weight gradient alone, loss-scaled fp16 with fp32 norm weights beside it
        _clip("head", "fp16", 1, 128256 * 4096, vectors=3, vector=4096, scaled=1024.0),
        # a model's fp32 gradients
        _clip("model", "fp32", 288, 3670016, vectors=65, vector=4096),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    if rng.random() < 0.6:
        dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        vocab = spread(1000, 160000)
        rows = min(spread(1, 8192), max(1, (1 << 27) // vocab))
        capped = rng.random() < 0.25
        return _sample(None, rows, vocab, dtype, rng.choice(["own", "chat", "nucleus", "minp", "mixed"]),
                       pitch=vocab + rng.choice([0, 0, 1, 64]), softcap=30.0 if capped else 0.0,
                       scale=0.5 if capped else 1.0, masked=rng.choice([0.0, 0.0, 0.3]))
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    tensors = spread(1, 500)
    elements = min(spread(100, 1 << 25), (1 << 28) // tensors)
    return _clip(None, dtype, tensors, elements, spread=rng.random() < 0.5, vectors=rng.choice([0, 5, 33]),
                 vector=spread(64, 8192), over=rng.choice([0.5, 2.0, 10.0]),
                 scaled=rng.choice([1.0, 1024.0]) if dtype == "fp16" else 1.0)


# ------------------------------------------------------------------ inputs ----

def _settings(case, g):
    """The requests' settings: fp32 / int32 arrays, or None where no request asks for one."""
    n, kind = case["rows"], case["settings"]
    if kind == "own":
        return dict(temperature=None, top_k=None, top_p=None, min_p=None)

    def uniform(lo, hi):
        return lo + (hi - lo) * torch.rand(n, generator=g, device="cuda")

    t = uniform(0.6, 1.1)
    k = uniform(20, 100).to(torch.int32)
    p = uniform(0.8, 0.97)
    m = uniform(0.02, 0.1)
    if kind == "chat":
        return dict(temperature=t, top_k=k, top_p=p, min_p=None)
    if kind == "nucleus":
        return dict(temperature=t, top_k=None, top_p=p, min_p=None)
    if kind == "minp":
        return dict(temperature=t, top_k=None, top_p=None, min_p=m)
    # mixed: greedy, unfiltered, top-k, top-p, both, min-p in turn, from a random start
    which = (torch.arange(n, device="cuda") + torch.randint(6, (1,), generator=g, device="cuda")) % 6
    return dict(temperature=torch.where(which == 0, 0.0, t),
                top_k=torch.where((which == 2) | (which == 4), k, 0),
                top_p=torch.where((which == 3) | (which == 4), p, 1.0),
                min_p=torch.where(which == 5, m, 0.0))


def _sizes(case):
    n, m = case["tensors"], case["elements"]
    if not case["spread"]:
        return [m] * n
    return [max(1, int(m ** ((i % 7 + 1) / 7.0))) + i % 3 for i in range(n)]


def _logits(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    n, v, pitch = case["rows"], case["vocab"], case["pitch"]
    # a broad body of another width in every row, and a few dozen plausible tokens above it
    x = torch.randn(n, pitch, generator=g, device="cuda")
    x *= 1.5 + 1.5 * torch.rand(n, 1, generator=g, device="cuda")
    at = torch.randint(v, (n, 24), generator=g, device="cuda")
    x.scatter_reduce_(1, at, 4 + 10 * torch.rand(n, 24, generator=g, device="cuda"), "amax")
    if case["scale"] != 1.0:
        x *= 2.0
    if case["masked"]:
        rows = torch.rand(n, 1, generator=g, device="cuda") < case["masked"]
        x.masked_fill_(rows & (torch.rand(n, pitch, generator=g, device="cuda") < 0.9), -math.inf)
    return x.to(DTYPES[case["dtype"]]), g


def _gradients(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    sizes = _sizes(case)
    flat = torch.randn(sum(sizes), generator=g, device="cuda")
    # from tensor to tensor the gradients' size differs by orders of magnitude; in fp16 it has to
    # stay in the type's range after the loss scale is taken off
    ratio, middle = (0.5, 1e-2) if case["dtype"] == "fp16" else (2.0, 1e-4)
    width = torch.exp(ratio * torch.randn(len(sizes), generator=g, device="cuda")) * middle
    flat *= width.repeat_interleave(torch.tensor(sizes, device="cuda"))
    flats = [flat.to(DTYPES[case["dtype"]]) if case["scaled"] == 1.0 else
             (flat * case["scaled"]).to(DTYPES[case["dtype"]])]
    del flat
    if case["vectors"]:
        flats.append(torch.randn(case["vectors"] * case["vector"], generator=g, device="cuda")
                     * (1e-3 * case["scaled"]))
    return flats


def prepare(case, seed):
    if case["op"] == "sample":
        x, g = _logits(case, seed)
        s = dict(case=case, logits=x[:, :case["vocab"]], **_settings(case, g))
        s["uniforms"] = torch.rand(case["rows"], generator=g, device="cuda", dtype=torch.float64)
        if own:
            import gradient_row_online_gb300 as pkg
            s["sampler"] = pkg.HeadSampler(softcap=case["softcap"], logits_scale=case["scale"])
        return s
    flats = _gradients(case, seed)
    outs = [torch.empty_like(f) for f in flats]
    sizes = [_sizes(case), [case["vector"]] * case["vectors"]]
    norm = math.sqrt(sum(float(f.float().square().sum(dtype=torch.float64)) for f in flats))
    s = dict(case=case, flats=flats, outs=outs, inv_scale=1.0 / case["scaled"],
             max_norm=norm / case["scaled"] / case["over"],
             grads=[t for f, z in zip(flats, sizes) for t in f.split(z)])
    if own:
        import gradient_row_online_gb300 as pkg
        s["clipper"] = pkg.GradClipper(s["grads"], [t for f, z in zip(outs, sizes) for t in f.split(z)])
    return s


# ------------------------------------------------------------- plain forms ----

def _plain_sample(s):
    case = s["case"]
    x = s["logits"].float()
    x = torch.where(x != x, -math.inf, x)
    allowed = x != -math.inf
    top = x.amax(1, keepdim=True)
    cap, scale = case["softcap"], case["scale"]
    z, zm = (x, top) if cap == 0 else (torch.tanh(x * (1.0 / cap)) * cap, torch.tanh(top * (1.0 / cap)) * cap)
    n = x.shape[0]
    t = s["temperature"] if s["temperature"] is not None else torch.ones(n, device=x.device)
    k = torch.full_like(t, scale * LOG2E)
    c = k / t
    greedy = ~torch.isfinite(c)
    c = torch.where(greedy, k, c)
    d = torch.where(z == zm, 0.0, (z - zm) * c[:, None])
    e = torch.where(allowed, torch.exp2(d), 0.0)
    w = torch.round(e * UNIT).to(torch.int64)
    column = torch.arange(x.shape[1], device=x.device)
    best = torch.where(x == top, column, x.shape[1]).amin(1, keepdim=True)
    keep = ~greedy[:, None] | (column == best)
    if s["top_k"] is not None or s["top_p"] is not None:
        order = x.sort(dim=1, descending=True, stable=True).indices
        ws = w.gather(1, order)
        first = s["top_k"] if s["top_k"] is not None else torch.zeros_like(t, dtype=torch.int32)
        first = torch.where(greedy, 1, torch.where(first <= 0, x.shape[1], first))
        ks = column < first[:, None]
        ws = ws * ks
        if s["top_p"] is not None:
            before = ws.cumsum(1) - ws
            ks &= (before.double() < (s["top_p"].double() * ws.sum(1).double())[:, None]) | (column == 0)
        keep = torch.zeros_like(allowed).scatter_(1, order, ks)
    if s["min_p"] is not None:
        keep &= e >= s["min_p"][:, None]
    w = torch.where(keep, w, 0)
    total = w.sum(1)
    target = torch.minimum(torch.floor(s["uniforms"] * total.double()).to(torch.int64), total - 1)
    token = (w.cumsum(1) <= target[:, None]).sum(1)
    empty = total == 0
    at = torch.where(empty, 0, token)[:, None]
    zt = (z.gather(1, at) - zm).squeeze(1)
    own_mass = torch.where(allowed, torch.exp((z - zm) * scale), 0.0).sum(1)
    logprob = zt * scale - torch.log(own_mass)
    drawn = d.gather(1, at).squeeze(1) * math.log(2.0) - torch.log((total.double() / UNIT).float())
    return dict(token=torch.where(empty, -1, token), logprob=torch.where(empty, 0.0, logprob),
                draw_logprob=torch.where(empty, 0.0, drawn), kept=(w > 0).sum(1).to(torch.int32))


def _plain_clip(s):
    wide = [f.float() for f in s["flats"]]
    norm = s["inv_scale"] * torch.sqrt(torch.stack([f.square().sum() for f in wide]).sum())
    factor = s["inv_scale"] * torch.where(norm > s["max_norm"], s["max_norm"] / norm, 1.0)
    return dict(stats=torch.stack([norm, factor]),
                out=[(f * factor).to(g.dtype) for f, g in zip(wide, s["flats"])])


def run(s):
    if s["case"]["op"] == "sample":
        if not own:
            return _plain_sample(s)
        token, logprob, drawn, kept = s["sampler"](s["logits"], s["uniforms"], temperature=s["temperature"],
                                                   top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
        return dict(token=token, logprob=logprob, draw_logprob=drawn, kept=kept)
    if not own:
        return _plain_clip(s)
    return dict(stats=s["clipper"](s["max_norm"], s["inv_scale"]), out=s["outs"])


def work(case):
    if case["op"] == "sample":
        n, v = case["rows"], case["vocab"]
        # the logits; a uniform, the settings in use; a token, two log-probs and a count
        return dict(bytes=n * (v * BYTES[case["dtype"]] + 8 + 16 + 8 + 12), flops=4 * n * v)
    n, m = sum(_sizes(case)), case["vectors"] * case["vector"]
    return dict(bytes=2 * (n * BYTES[case["dtype"]] + 4 * m) + 8, flops=3 * (n + m))


# -------------------------------------------------------- the 64-bit values ----

def exact(case, seed):
    """The definitions in 64 bits, a row (a tensor) at a time."""
    if case["op"] == "clip":
        flats = _gradients(case, seed)
        norm32 = math.sqrt(sum(float(f.float().square().sum(dtype=torch.float64)) for f in flats))
        max_norm = norm32 / case["scaled"] / case["over"]
        norm = math.sqrt(sum(float(p.double().pow(2).sum()) for f in flats for p in f.split(1 << 26))) / case["scaled"]
        factor = min(1.0, max_norm / norm) / case["scaled"]
        return dict(stats=torch.tensor([norm, factor], dtype=torch.float64),
                    out=[f.double() * factor for f in flats])
    logits, g = _logits(case, seed)
    settings = _settings(case, g)
    n, v, cap, scale = case["rows"], case["vocab"], case["softcap"], case["scale"]
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    lists = {key: None if a is None else a.tolist() for key, a in settings.items()}
    tokens, logprobs, draws = [], [], []
    for i in range(n):
        x = logits[i, :v].double()
        z = cap * torch.tanh(x / cap) if cap else x
        t = 1.0 if lists["temperature"] is None else lists["temperature"][i]
        mass = torch.exp((z - z.max()) * (scale / t if t else scale)).masked_fill(x == -math.inf, 0.0)
        model = torch.exp((z - z.max()) * scale).masked_fill(x == -math.inf, 0.0)
        weight = torch.round(mass * UNIT)
        least = torch.zeros_like(x, dtype=torch.bool)
        k = 0 if lists["top_k"] is None else lists["top_k"][i]
        k = 1 if not t else k
        p = 1.0 if lists["top_p"] is None else lists["top_p"][i]
        if k or p < 1:
            falling = torch.argsort(-x, stable=True)[:k or v]
            above = torch.cumsum(weight[falling], 0)
            count = 1 + torch.searchsorted(above, p * above[-1:]) if p < 1 else falling.numel()
            least[falling[:count]] = True
        else:
            least[:] = True
        if lists["min_p"] is not None:
            least &= mass >= lists["min_p"][i]
        inside = torch.cumsum(weight * least, 0)
        at = torch.searchsorted(inside, torch.floor(u[i] * inside[-1]), right=True).clamp(max=v - 1)
        empty = inside[-1] == 0
        tokens.append(torch.where(empty, -1, at))
        logprobs.append(torch.where(empty, 0.0, torch.log(model[at] / model.sum())))
        draws.append(torch.where(empty, 0.0, torch.log(mass[at] / (mass * least).sum())))
    stack = lambda a: torch.stack(a).reshape(n)  # noqa: E731
    return dict(token=stack(tokens), logprob=stack(logprobs), draw_logprob=stack(draws), kept=None)
