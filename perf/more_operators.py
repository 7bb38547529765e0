"""What is measured of the operators that stand around an 8-bit head: the head's product with one
scale for each block of 128 (its logits, and a training step's logits and both gradients), the
selection of a beam search over beams and vocabulary, and the reordering of the beams' states.

`run` computes them in plain torch operations, or (`own`) through the library's public entry points.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16, "int8": torch.int8}
BYTES = {"fp32": 4, "bf16": 2, "fp16": 2, "int8": 1}
# the 8-bit types, and the largest value of each
FP8 = {"e4m3": (torch.float8_e4m3fn, 448.0), "e5m2": (torch.float8_e5m2, 57344.0)}
LEAST = 2.0 ** -126  # the smallest scale


def _logits(name, tokens, width, vocab, dtype="bf16", out="bf16"):
    case = dict(op="logits", tokens=tokens, width=width, vocab=vocab, dtype=dtype, out=out)
    return dict(case, name=name) if name else case


def _train(name, tokens, width, vocab, dtype="bf16", master="bf16", grads="e4m3"):
    case = dict(op="train", tokens=tokens, width=width, vocab=vocab, dtype=dtype, master=master, grads=grads)
    return dict(case, name=name) if name else case


def _beam(name, requests, beams, keep, vocab, dtype="bf16", pitch=0, softcap=0.0, scale=1.0, first=False,
          ended=0.0, stay=False, masked=0.0):
    case = dict(op="beam", requests=requests, beams=beams, keep=keep, vocab=vocab, dtype=dtype, pitch=pitch or vocab,
                softcap=softcap, scale=scale, first=first, ended=ended, stay=stay, masked=masked)
    return dict(case, name=name) if name else case


def _reorder(name, requests, beams, tensors, heads, positions, width, dtype="bf16", ranged=True, inplace=True):
    case = dict(op="reorder", requests=requests, beams=beams, tensors=tensors, heads=heads, positions=positions,
                width=width, dtype=dtype, ranged=ranged, inplace=inplace)
    return dict(case, name=name) if name else case


def listed():
    return [
        # one interactive request's next token: the weights' bytes and the call's latency
        _logits("one token", 1, 4096, 32000),
        # a decoding batch over a large vocabulary: still the weights' bytes
        _logits("decoding batch", 48, 4096, 128256),
        # a ragged prefill with an odd vocabulary and a width that ends inside a block
        _logits("odd prefill", 333, 2056, 32003, dtype="fp16", out="fp32"),
        # scoring long prompts: the tensor cores
        _logits("scoring", 8192, 4096, 32000),
        # a probe's training step, odd in every size, fp32 hidden states and weights
        _train("small step", 200, 1000, 5003, dtype="fp32", master="fp32", grads="e5m2"),
        # the head of a training step: weights requantised after the optimiser, three products
        _train("training step", 4096, 4096, 128256),
        # the first step of one request: its beams are the same, all but the first are dead
        _beam("first beams", 1, 4, 8, 32000, first=True),
        # a batch with some hypotheses ended, fp32 logits with an odd vocabulary, some under a grammar
        _beam("ended beams", 24, 5, 5, 32003, dtype="fp32", ended=0.3, stay=True, masked=0.25),
        # a full batch of a capped and scaled head with a padded vocabulary
        _beam("full beams", 256, 8, 16, 151936, pitch=152064, softcap=30.0, scale=0.5),
        # one request's key-value caches, a short answer so far
        _reorder("short answer", 1, 4, 32, 8, 512, 128),
        # states of fixed size and odd shape, moved to other buffers
        _reorder("odd states", 7, 5, 24, 33, 0, 77, dtype="fp32", ranged=False, inplace=False),
        # a batch's caches: long answers to long prompts
        _reorder("long answers", 16, 4, 16, 8, 2048, 128),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    kind = rng.random()
    if kind < 0.35:
        width, vocab = spread(256, 8192), spread(1000, 160000)
        if width * vocab > 1 << 29:
            vocab = (1 << 29) // width
        most = (1 << 40) // (width * vocab)
        return _logits(None, min(spread(1, 8192), most), width, vocab, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                       out=rng.choice(["bf16", "bf16", "fp16", "fp32"]))
    if kind < 0.5:
        width, vocab = spread(200, 4096), spread(1000, 128256)
        return _train(None, min(spread(16, 4096), (1 << 38) // (width * vocab)), width, vocab,
                      dtype=rng.choice(["bf16", "fp16", "fp32"]), master=rng.choice(["bf16", "fp32"]),
                      grads=rng.choice(["e4m3", "e5m2"]))
    if kind < 0.8:
        vocab, beams = spread(1000, 160000), rng.choice([1, 2, 3, 4, 5, 8, 16])
        requests = min(spread(1, 256), max(1, (1 << 28) // (vocab * beams)))
        keep = rng.choice([beams, 2 * beams])
        capped = rng.random() < 0.3
        return _beam(None, requests, beams, keep, vocab, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                     pitch=vocab + rng.choice([0, 0, 1, 64]), softcap=30.0 if capped else 0.0,
                     scale=0.5 if capped else 1.0, first=rng.random() < 0.2, ended=rng.choice([0.0, 0.0, 0.3]),
                     stay=keep == beams and rng.random() < 0.5, masked=rng.choice([0.0, 0.0, 0.3]))
    beams, heads, width = rng.choice([2, 3, 4, 8, 16]), spread(1, 32), rng.choice([64, 80, 96, 128, 37])
    requests, tensors = spread(1, 64), spread(1, 32)
    positions = min(spread(8, 4096), max(4, (1 << 30) // (requests * beams * tensors * heads * width)))
    return _reorder(None, requests, beams, tensors, heads, positions, width, dtype=rng.choice(["bf16", "fp16", "int8", "fp32"]),
                    ranged=rng.random() < 0.7, inplace=rng.random() < 0.6)


# ------------------------------------------------------------------ inputs ----

def _hidden(case, g):
    # normalised hidden states: some channels are far wider than the others
    n, d = case["tokens"], case["width"]
    width = torch.where(torch.rand(d, generator=g, device="cuda") < 0.01, 12.0, 1.0)
    return (torch.randn(n, d, generator=g, device="cuda") * width).to(DTYPES[case["dtype"]])


def _weight(case, g):
    v, d = case["vocab"], case["width"]
    # rare tokens' rows are smaller
    row = 0.3 + 0.7 * torch.rand(v, 1, generator=g, device="cuda")
    return torch.randn(v, d, generator=g, device="cuda").mul_(row * d ** -0.5)


def _head_inputs(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    s = dict(case=case, hidden=_hidden(case, g))
    w = _weight(case, g)
    if case["op"] == "logits":
        # a checkpoint's weights: 8-bit values, one fp32 scale for each 128 x 128
        s["weight"], s["scales"] = _quantised(w, "e4m3", 128)
        return s
    s["weight"] = w.to(DTYPES[case["master"]])
    # the loss's gradient, from rows of plausible logits: softmax less the label, over the tokens
    n, v = case["tokens"], case["vocab"]
    x = torch.randn(n, v, generator=g, device="cuda").mul_(2.5)
    label = torch.randint(v, (n, 1), generator=g, device="cuda")
    x.scatter_(1, label, 9.0)
    x.sub_(x.amax(1, keepdim=True)).exp_()
    x.mul_(1.0 / (n * x.sum(1, keepdim=True)))
    x.scatter_add_(1, label, torch.full((n, 1), -1.0 / n, device="cuda"))
    if case["dtype"] == "fp16":
        x *= 1024.0  # the loss's scale
    s["grad"] = x.to(DTYPES[case["dtype"]])
    return s


def _beam_inputs(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    r, b, v, pitch = case["requests"], case["beams"], case["vocab"], case["pitch"]
    n = r * b
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
    scores = -20.0 - 3.0 * torch.rand(r, b, generator=g, device="cuda")
    if case["first"]:
        x = x.view(r, b, pitch)[:, :1].expand(r, b, pitch).reshape(n, pitch)
        scores = torch.full_like(scores, -math.inf)
        scores[:, 0] = 0.0
    ended = torch.rand(r, b, generator=g, device="cuda") < case["ended"] if case["ended"] else None
    return dict(case=case, logits=x.to(DTYPES[case["dtype"]])[:, :v], scores=scores, ended=ended)


def _reorder_inputs(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    r, b, p = case["requests"], case["beams"], case["positions"]
    shape = (r * b, case["heads"]) + ((p,) if p else ()) + (case["width"],)
    kind = DTYPES[case["dtype"]]
    if case["dtype"] == "int8":
        states = [torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=kind) for _ in range(case["tensors"])]
    else:
        states = [torch.randn(shape, generator=g, device="cuda").to(kind) for _ in range(case["tensors"])]
    parents = torch.randint(b, (r, b), generator=g, device="cuda", dtype=torch.int32)
    if case["inplace"]:
        # as the selection gives them to states that stay where they are: a beam that goes on keeps its place
        column = torch.arange(b, device="cuda", dtype=torch.int32)
        goes_on = torch.rand(r, b, generator=g, device="cuda") < 0.6
        goes_on |= column == parents[:, :1]
        pick = torch.where(goes_on, torch.rand(r, b, generator=g, device="cuda"), -1.0)
        order = pick.argsort(dim=1, descending=True)
        of = order.gather(1, parents.long() % goes_on.sum(1, keepdim=True))
        parents = torch.where(goes_on, column, of.to(torch.int32))
    begin = end = None
    if case["ranged"] and p:
        begin = (p * (0.25 + 0.5 * torch.rand(r, generator=g, device="cuda"))).to(torch.int32)
        end = begin + (p * 0.25 * torch.rand(r, generator=g, device="cuda")).to(torch.int32) + 1
    # the second buffers hold the prompts as well
    outs = states if case["inplace"] else [t.clone() for t in states]
    return dict(case=case, states=states, outs=outs, parents=parents, begin=begin, end=end)


INPUTS = dict(logits=_head_inputs, train=_head_inputs, beam=_beam_inputs, reorder=_reorder_inputs)


def prepare(case, seed):
    s = INPUTS[case["op"]](case, seed)
    if own:
        import gradient_row_online_gb300 as pkg
        if case["op"] == "logits":
            s["head"] = pkg.Fp8Head.from_quantized(s["weight"], s["scales"])
        elif case["op"] == "train":
            s["head"] = pkg.Fp8Head(s["weight"], train=True, grads=case["grads"])
        elif case["op"] == "beam":
            s["selector"] = pkg.BeamSelector(case["beams"], case["keep"], softcap=case["softcap"], logits_scale=case["scale"],
                                             eos=2 if case["ended"] else None, stay=case["stay"])
        else:
            s["reorder"] = pkg.StateReorder(s["states"], case["beams"], None if case["inplace"] else s["outs"],
                                            axis=2 if case["positions"] else None)
    return s


# ------------------------------------------------------------- plain forms ----

def _quantised(x, kind, rows):
    """`x` in 8 bits with one scale for each `rows` x 128 elements: the codes, and the scales, a row of
    them for each `rows` rows of x."""
    n, k = x.shape
    dtype, top = FP8[kind]
    t = torch.nn.functional.pad(x.float(), (0, -k % 128, 0, -n % rows))
    t = t.view(t.shape[0] // rows, rows, t.shape[1] // 128, 128)
    size = t.abs().amax((1, 3), keepdim=True)
    scale = torch.where(torch.isfinite(size), torch.clamp(size * (1.0 / top), min=LEAST), math.nan)
    q = (t * torch.reciprocal(scale)).to(dtype)
    return q.view(q.shape[0] * rows, -1)[:n, :k].contiguous(), scale.view(scale.shape[0], scale.shape[2])


def _values(q, scales, rows):
    """What the codes stand for."""
    n, k = q.shape
    wide = scales.repeat_interleave(128, 1)[:, :k]
    return q.float() * (wide if rows == 1 else wide.repeat_interleave(rows, 0)[:n])


def _coded(x, kind, rows):
    return _values(*_quantised(x, kind, rows), rows)


def _plain_logits(s):
    x = _coded(s["hidden"], "e4m3", 1)
    return (x @ _values(s["weight"], s["scales"], 128).t()).to(DTYPES[s["case"]["out"]])


def _plain_train(s):
    case = s["case"]
    weight = _coded(s["weight"], "e4m3", 128)
    logits = (_coded(s["hidden"], "e4m3", 1) @ weight.t()).to(s["hidden"].dtype)
    grad_hidden = (_coded(s["grad"], case["grads"], 1) @ weight).to(s["hidden"].dtype)
    del weight
    # over the tokens: the gradient in 1 x 128 along them, the hidden states in 128 x 128
    grad_weight = _coded(s["grad"].t(), case["grads"], 1) @ _coded(s["hidden"].t(), "e4m3", 128).t()
    return dict(logits=logits, grad_hidden=grad_hidden, grad_weight=grad_weight.to(s["weight"].dtype))


def _plain_beam(s):
    case = s["case"]
    r, b, k, v, cap = case["requests"], case["beams"], case["keep"], case["vocab"], case["softcap"]
    x = s["logits"].double()
    z = torch.tanh(x / cap) * cap if cap else x
    top = z.amax(1, keepdim=True)
    # a row in which nothing is allowed has no candidates
    d = torch.where(z == -math.inf, -math.inf, (z - top) * case["scale"])
    mass = torch.exp(d.float()).sum(1, keepdim=True, dtype=torch.float64)
    before = s["scores"].double().view(r * b, 1)
    score = torch.where(d == -math.inf, -math.inf, before + (d - torch.log(mass)))
    column = torch.arange(v, device=x.device)
    if s["ended"] is not None:  # one candidate: itself, at the token that ended it
        score = torch.where(s["ended"].view(r * b, 1), torch.where(column == 2, before, -math.inf), score)
    score = score.view(r, b * v)
    score, at = (t[:, :k] for t in score.sort(dim=1, descending=True, stable=True))
    none = score == -math.inf
    parent = torch.where(none, -1, at // v)
    token = torch.where(none, -1, at % v)
    ended = torch.zeros_like(none)
    if s["ended"] is not None:
        ended = ~none & (s["ended"].gather(1, parent.clamp(min=0)) | (token == 2))
    if case["stay"]:  # the first child of a beam takes its place, the others fill the free ones
        earlier = (parent[:, :, None] == parent[:, None, :]).tril(-1).any(2)
        first = ~earlier & ~none
        taken = torch.zeros(r, k + 1, dtype=torch.bool, device=x.device).scatter_(1, torch.where(first, parent, k), True)[:, :k]
        free = taken.to(torch.int8).argsort(dim=1, stable=True)
        place = torch.where(first, parent, free.gather(1, ((~first).cumsum(1) - 1).clamp(min=0)))
        score, parent, token, ended = (torch.empty_like(t).scatter_(1, place, t) for t in (score, parent, token, ended))
    return dict(scores=score.float(), parents=parent.to(torch.int32), tokens=token, ended=ended)


def _plain_reorder(s):
    case = s["case"]
    r, b, p = case["requests"], case["beams"], case["positions"]
    rows = (s["parents"] + torch.arange(r, device="cuda")[:, None] * b).view(-1)
    if s["begin"] is None:
        return [o.copy_(t[rows]) for t, o in zip(s["states"], s["outs"])]
    at = torch.arange(p, device="cuda")
    inside = (at >= s["begin"][:, None]) & (at < s["end"][:, None])
    inside = inside.repeat_interleave(b, 0)[:, None, :, None]
    return [o.copy_(torch.where(inside, t[rows], o)) for t, o in zip(s["states"], s["outs"])]


PLAIN = dict(logits=_plain_logits, train=_plain_train, beam=_plain_beam, reorder=_plain_reorder)


def run(s):
    case = s["case"]
    if not own:
        return PLAIN[case["op"]](s)
    if case["op"] == "logits":
        return s["head"].logits(s["hidden"], dtype=DTYPES[case["out"]])
    if case["op"] == "train":
        head = s["head"]
        head.set_weight(s["weight"])
        logits = head.logits(s["hidden"])
        grad_hidden, grad_weight = head.backward(s["grad"], s["hidden"])
        return dict(logits=logits, grad_hidden=grad_hidden, grad_weight=grad_weight)
    if case["op"] == "beam":
        scores, parents, tokens, ended = s["selector"](s["logits"], s["scores"], s["ended"])
        return dict(scores=scores, parents=parents, tokens=tokens, ended=ended)
    return s["reorder"](s["parents"], s["begin"], s["end"])


def work(case):
    if case["op"] in ("logits", "train"):
        n, d, v = case["tokens"], case["width"], case["vocab"]
        scales = 4 * -(-v // 128) * -(-d // 128)
        if case["op"] == "logits":
            return dict(bytes=v * d + scales + n * d * BYTES[case["dtype"]] + n * v * BYTES[case["out"]], flops=2 * n * d * v)
        # weights, hidden states and the loss's gradient in; logits and both gradients out
        return dict(bytes=2 * v * d * BYTES[case["master"]] + 2 * n * (d + v) * BYTES[case["dtype"]], flops=6 * n * d * v)
    if case["op"] == "beam":
        # the beams that can have children, once; scores in, and scores, parents, tokens and ends out
        live = case["requests"] * (1 if case["first"] else case["beams"]) * (1 - case["ended"])
        return dict(bytes=live * case["vocab"] * BYTES[case["dtype"]] + case["requests"] * (5 * case["beams"] + 17 * case["keep"]),
                    flops=4 * live * case["vocab"])
    # of b beams, each drawn again at random, 1 - (1 - 1 / b)^b are read; all are written, in place those that change
    b, p = case["beams"], case["positions"]
    row = case["heads"] * max(1, p) * case["width"] * BYTES[case["dtype"]] * case["tensors"]
    if case["ranged"] and p:
        row *= 0.125
    stay = 0.4 + 0.6 * b if case["inplace"] else 0
    moved = b - stay
    drawn = stay or b
    return dict(bytes=case["requests"] * row * (moved + drawn * (1 - (1 - 1 / drawn) ** moved)), flops=0)


# -------------------------------------------------------- the 64-bit values ----

def _code(x, kind, rows):
    """The definition of the 8-bit form, its values in 64 bits: for each rows x 128 elements an fp32 scale, their largest
    magnitude times the fp32 value of 1 / top (2^-126 at least), and each element times the fp32 inverse of the scale,
    in fp32, rounded to the 8-bit type."""
    dtype, top = FP8[kind]
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    step = rows if rows > 1 else max(1, x.shape[0])
    for i in range(0, x.shape[0], step):
        for j in range(0, x.shape[1], 128):
            t = x[i:i + step, j:j + 128].float()
            size = t.abs().max() if rows > 1 else t.abs().max(1, keepdim=True).values
            scale = torch.maximum(size * torch.tensor(1.0 / top, dtype=torch.float32, device=x.device),
                                  torch.tensor(LEAST, dtype=torch.float32, device=x.device))
            out[i:i + step, j:j + 128] = (t * (1.0 / scale)).to(dtype).double() * scale.double()
    return out


def _exact_head(case, seed):
    s = _head_inputs(case, seed)
    x = s["hidden"]
    if case["op"] == "logits":
        w = s["weight"].double()
        for i in range(s["scales"].shape[0]):
            for j in range(s["scales"].shape[1]):
                w[128 * i:128 * i + 128, 128 * j:128 * j + 128] *= s["scales"][i, j].double()
        return torch.einsum("nd,vd->nv", _code(x, "e4m3", 1), w)
    w = _code(s["weight"], "e4m3", 128)
    logits = torch.einsum("nd,vd->nv", _code(x, "e4m3", 1), w)
    grad_hidden = torch.einsum("nv,vd->nd", _code(s["grad"], case["grads"], 1), w)
    del w
    turned = _code(s["grad"].t(), case["grads"], 1)
    grad_weight = torch.einsum("vn,dn->vd", turned, _code(x.t(), "e4m3", 128))
    return dict(logits=logits, grad_hidden=grad_hidden, grad_weight=grad_weight)


def _exact_beam(case, seed):
    """The scores: of every request, its candidates' in falling order."""
    if case["stay"]:
        return None  # where each stands goes by the parents
    s = _beam_inputs(case, seed)
    r, b, k, cap = case["requests"], case["beams"], case["keep"], case["softcap"]
    scores = torch.full((r, k), -math.inf, dtype=torch.float64, device="cuda")
    for i in range(r):
        found = []
        for j in range(b):
            if s["ended"] is not None and bool(s["ended"][i, j]):
                found.append(s["scores"][i, j:j + 1].double())
                continue
            x = s["logits"][i * b + j].double()
            z = case["scale"] * (cap * torch.tanh(x / cap) if cap else x)
            found.append((s["scores"][i, j].double() + torch.log_softmax(z, 0)).nan_to_num(nan=-math.inf).topk(min(k, x.numel())).values)
        best = torch.cat(found).sort(descending=True).values[:k]
        scores[i, :best.numel()] = best
    return dict(scores=scores, parents=None, tokens=None, ended=None)


def _exact_reorder(case, seed):
    s = _reorder_inputs(case, seed)
    b = case["beams"]
    parents = s["parents"].tolist()
    outs = [t.clone() for t in s["states"]]
    for i, row in enumerate(parents):
        some = slice(None) if s["begin"] is None else slice(int(s["begin"][i]), int(s["end"][i]))
        for j, parent in enumerate(row):
            for t, o in zip(s["states"], outs):
                if s["begin"] is None:
                    o[i * b + j] = t[i * b + parent]
                else:
                    o[i * b + j, :, some] = t[i * b + parent, :, some]
    return outs


def exact(case, seed):
    return dict(logits=_exact_head, train=_exact_head, beam=_exact_beam, reorder=_exact_reorder)[case["op"]](case, seed)
