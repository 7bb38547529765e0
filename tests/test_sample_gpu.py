"""headloss_sample against its definition, twice.

`definition` is the definition in elementary torch operations on the GPU: integer
weights from fp32 logits, so tokens and kept counts have to be equal to the bit.

`row_reference` is the definition in 64 bits (numpy).  There the library's cuts lie
within a relative TAU of the real ones, and the token within the indexes that
moving every cut (top-p's target, min-p's threshold, the drawn target) by TAU
spans.  TAU: an exponent d of up to 31 carries the roundings of a difference and
a product, 2^-23 * 31 * ln 2 relative in 2^d, the exponential two ulps more,
and the integer grid 2^-31 of the largest weight a token.  Log-probs are held to
2e-6 + 2e-6 |log p|: differences and sums in fp32 of magnitudes below 64, each
rounding 2^-24 relative, and a logarithm."""
import math

import numpy as np
import pytest
import torch

import gradient_row_online_gb300 as pkg
from gradient_row_online_gb300 import headloss as hlb

pytestmark = pytest.mark.gpu

LOG2E = 1.4426950408889634
TAU = 4e-6
INF = math.inf
DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}


def row_reference(x, u, t=1.0, k=0, p=1.0, m=0.0, cap=0.0, s=1.0):
    """A row in 64 bits: the range of tokens, log p and d ln 2 by token, the range of
    log W and of the kept count; None for a row without a token."""
    x = np.where(np.isnan(x), -INF, x.astype(np.float64))
    if not (x > -INF).any():
        return None
    top = x.max()
    z = cap * np.tanh(x / cap) if cap else x
    zm = cap * math.tanh(top / cap) if cap else top
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        diff = np.where(z == zm, 0.0, z - zm)
        if t == 0 or s * LOG2E / t > 3.4e38:
            t, k = 1.0, 1
        c = s * LOG2E / t
        d = np.where(x > -INF, diff * c, -INF)
        model = np.where(x > -INF, diff * s, -INF)
    w = np.rint(2.0 ** 30 * 2.0 ** d)
    order = np.lexsort((np.arange(x.size), -x))
    if 0 < k < x.size:
        order = order[:k]
    above = np.concatenate([[0.0], np.cumsum(w[order])])
    answers = []
    for f in (1 - TAU, 1.0, 1 + TAU):
        n = order.size
        if p < 1:
            n = max(1, int(np.searchsorted(above[:-1], p * above[-1] * f, side="left")))
        kept = np.zeros(x.size, bool)
        kept[order[:n]] = True
        kept &= 2.0 ** d >= min(m * f, 1.0)  # the largest logit always stays
        wk = np.where(kept, w, 0.0)
        W = wk.sum()
        cum = np.cumsum(wk)
        for g in (-TAU, 0.0, TAU):
            tt = min(max(math.floor(u * W + g * W), 0), W - 1)
            answers.append((int(np.searchsorted(cum, tt, side="right")), math.log(W / 2.0 ** 30),
                            int((wk > 0).sum())))
    lse = math.log(np.exp(model).sum())
    return dict(tokens=(min(a[0] for a in answers), max(a[0] for a in answers)), logprob=model - lse, d=d * math.log(2.0),
                logw=(min(a[1] for a in answers), max(a[1] for a in answers)), kept=(min(a[2] for a in answers),
                                                            max(a[2] for a in answers)))


def run(logits, u, cap=0.0, s=1.0, **settings):
    sampler = pkg.HeadSampler(softcap=cap, logits_scale=s)
    out = sampler(logits, u, **settings)
    err = sampler.device_error()
    return [o.cpu().numpy() for o in out], err


def definition(x, u, t, k, p, m, cap, s):
    """(tokens, kept counts) of the definition, in torch operations."""
    n, v = x.shape
    x = x.float() + 0.0
    x = torch.where(x != x, -INF, x)
    top = x.amax(1, keepdim=True)
    z, zm = (x, top) if cap == 0 else (torch.tanh(x * (1 / cap)) * cap, torch.tanh(top * (1 / cap)) * cap)
    one = torch.ones(n, device=x.device)
    c = (one * (s * LOG2E)) / (one if t is None else t)
    greedy = ~torch.isfinite(c)
    c = torch.where(greedy, s * LOG2E, c)
    k = torch.where(greedy, 1, torch.zeros_like(one, dtype=torch.int32) if k is None else k)
    k = torch.where(k <= 0, v, k)
    d = torch.where(z == zm, 0.0, (z - zm) * c[:, None])
    e = torch.where(x == -INF, 0.0, torch.exp2(d))
    w = torch.round(e * 2.0 ** 30).long()
    order = x.sort(dim=1, descending=True, stable=True).indices
    rank = torch.arange(v, device=x.device)
    keep = rank < k[:, None]
    ws = w.gather(1, order) * keep
    if p is not None:
        below = (ws.cumsum(1) - ws).double() < (p.double() * ws.sum(1).double())[:, None]
        keep &= (p >= 1)[:, None] | below | (rank == 0)
    keep = torch.zeros_like(keep).scatter_(1, order, keep)
    if m is not None:
        keep &= e >= m[:, None]
    w = w * keep
    W = w.sum(1)
    target = torch.minimum(torch.floor(u * W.double()).long(), W - 1)
    token = (w.cumsum(1) <= target[:, None]).sum(1)
    return torch.where(W == 0, -1, token).cpu().numpy(), (w > 0).sum(1).cpu().numpy()


def check(logits, u, cap=0.0, s=1.0, t=None, k=None, p=None, m=None):
    """Every row of a call against both references."""
    n = logits.shape[0]

    def dev(a, dtype):
        return None if a is None else torch.as_tensor(a, dtype=dtype).expand(n).contiguous().cuda()

    given = dict(temperature=dev(t, torch.float32), top_k=dev(k, torch.int32),
                 top_p=dev(p, torch.float32), min_p=dev(m, torch.float32))
    (tok, lp, dlp, kept), err = run(logits, u, cap, s, **given)
    assert err == 0
    want, count = definition(logits, u, *given.values(), cap, s)
    assert np.array_equal(tok, want), (tok, want)
    assert np.array_equal(kept, count), (kept, count)
    x = logits.float().cpu().numpy()
    host = {key: None if a is None else a.cpu().numpy() for key, a in given.items()}
    uu = u.cpu().numpy()
    for i in range(n):
        opt = {name: host[key][i] for name, key in
               (("t", "temperature"), ("k", "top_k"), ("p", "top_p"), ("m", "min_p"))
               if host[key] is not None}
        opt = {name: (int(v) if name == "k" else float(v)) for name, v in opt.items()}
        ref = row_reference(x[i], float(uu[i]), cap=cap, s=s, **opt)
        if ref is None:
            assert tok[i] == -1 and lp[i] == 0 and dlp[i] == 0 and kept[i] == 0
            continue
        j = int(tok[i])
        assert ref["tokens"][0] <= j <= ref["tokens"][1], (i, j, ref["tokens"])
        assert ref["kept"][0] <= kept[i] <= ref["kept"][1], (i, kept[i], ref["kept"])
        want = ref["logprob"][j]
        assert abs(lp[i] - want) <= 2e-6 + 2e-6 * abs(want), (i, lp[i], want)
        low, high = ref["d"][j] - ref["logw"][1], ref["d"][j] - ref["logw"][0]
        slack = 2e-6 + 2e-6 * abs(low)
        assert low - slack <= dlp[i] <= high + slack, (i, dlp[i], low, high)
    return tok


def noise(n, v, dtype, seed=0, sigma=3.0, pitch=None):
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(n, pitch or v, generator=g, device="cuda") * sigma
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    return x.to(DT[dtype])[:, :v], u


FILTERS = {"own": {}, "cool": dict(t=0.7), "hot": dict(t=1.8), "k": dict(k=40), "k1": dict(k=1),
           "kbig": dict(k=1500, t=0.9), "p": dict(p=0.9), "p0": dict(p=0.0), "ptiny": dict(p=1e-7),
           "m": dict(m=0.05), "m1": dict(m=1.0), "kp": dict(t=0.8, k=50, p=0.95),
           "kbigp": dict(k=1200, p=0.99), "kpm": dict(t=1.2, k=200, p=0.97, m=0.01),
           "pm": dict(p=0.98, m=0.001), "greedy": dict(t=0.0)}


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("name", FILTERS)
def test_every_filter(name, dtype):
    x, u = noise(24, 4099, dtype, seed=len(name))
    check(x, u, **FILTERS[name])


@pytest.mark.parametrize("v", [1, 2, 7, 8, 9, 31, 33, 255, 513, 1031, 8191, 32000, 32003])
@pytest.mark.parametrize("dtype,pad", [("bf16", 0), ("bf16", 1), ("fp16", 3), ("fp32", 0), ("fp32", 1)])
def test_sizes_and_strides(v, dtype, pad):
    x, u = noise(5, v, dtype, seed=v, pitch=v + pad)
    check(x, u)
    check(x, u, t=0.8, k=20, p=0.9)
    check(x, u, p=0.95)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_long_rows(dtype):
    x, u = noise(3, 151936, dtype, seed=5)
    check(x, u)
    check(x, u, t=0.9, k=64, p=0.9)
    check(x, u, p=0.9)
    check(x, u, k=20000, p=0.95)
    check(x, u, m=0.02)


def test_very_long_row():
    x, u = noise(1, 1_200_011, "bf16", seed=6, sigma=2.0)
    check(x, u, t=0.8, k=100, p=0.9)
    check(x, u, p=0.9)
    check(x, u)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("cap,s", [(30.0, 0.5), (5.0, 1.0), (0.0, 0.25)])
def test_softcap_and_scale(dtype, cap, s):
    x, u = noise(12, 5000, dtype, sigma=8.0)
    check(x, u, cap, s)
    check(x, u, cap, s, t=0.7, k=30, p=0.9)
    check(x, u, cap, s, p=0.9)


def test_ties_go_to_the_lowest_index():
    """A row of few distinct values: the cut falls inside long runs of equal logits."""
    g = torch.Generator().manual_seed(3)
    x = torch.randint(-2, 3, (16, 3001), generator=g).float()
    u = torch.rand(16, generator=g, dtype=torch.float64)
    for dtype in DT.values():
        xx, uu = x.to(dtype).cuda(), u.cuda()
        for f in (dict(k=17), dict(k=900), dict(p=0.3), dict(p=0.9), dict(k=700, p=0.5),
                  dict(k=2500, p=0.999), dict(t=0.0), dict(k=1), {}):
            check(xx, uu, **f)


def test_equal_rows_and_signed_zero():
    x = torch.zeros(4, 777)
    x[1] = -0.0
    x[2, ::2] = -0.0
    x[3] = -3.3e38
    u = torch.tensor([0.0, 0.5, 0.25, 0.999], dtype=torch.float64).cuda()
    for f in ({}, dict(k=10), dict(p=0.5), dict(t=0.0), dict(k=300, p=0.1)):
        check(x.bfloat16().cuda(), u, **f)
        check(x.cuda(), u, **f)


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
def test_masked_tokens(dtype):
    """-inf, the type's lowest value, +inf and NaN in masked places; rows with one token or none."""
    n, v = 12, 2050
    x, u = noise(n, v, dtype, seed=9)
    low = torch.finfo(DT[dtype]).min
    x[0] = -INF
    x[1] = -INF
    x[1, 77] = -5.0
    x[2, 100:] = low
    x[3, ::2] = float("nan")
    x[4] = float("nan")
    x[5, 3] = INF
    x[6, [9, 1000, 2049]] = INF
    x[7, :2049] = -INF
    x[8] = low
    x[9, 500:] = -INF
    x[10, ::3] = -INF
    x[10, 1::3] = float("nan")
    for f in ({}, dict(t=0.7, k=20, p=0.9), dict(p=0.9), dict(m=0.1), dict(t=0.0), dict(k=2),
              dict(k=1900), dict(k=1900, p=0.99)):
        tok = check(x, u, **f)
        assert tok[0] == -1 and tok[4] == -1 and tok[1] == 77 and tok[5] == 3 and tok[7] == 2049


def test_extreme_uniforms_and_temperatures():
    x, _ = noise(6, 3000, "bf16", seed=4)
    u = torch.tensor([0.0, 2.0 ** -53, 0.5, 1 - 2.0 ** -53, 0.999999, 1e-12], dtype=torch.float64).cuda()
    for t in (0.0, 1e-38, 1e-6, 1e-3, 50.0, 1e6, 3e38):
        check(x, u, t=t)
        check(x, u, t=t, k=10, p=0.8)


def test_settings_a_row():
    """Every row has its own settings; the rows do not depend on one another."""
    n, v = 36, 4000
    x, u = noise(n, v, "bf16", seed=12)
    t = torch.tensor([0.0, 0.5, 1.0, 1.3] * 9)
    k = torch.tensor([0, 1, 50, 2000, 5000, -1] * 6, dtype=torch.int32)
    p = torch.tensor([1.0, 0.9, 0.3] * 12)
    m = torch.tensor([0.0, 0.0, 0.1, 1.0, 0.0] * 8)[:n]
    whole = check(x, u, t=t, k=k, p=p, m=m)
    for i in (0, 7, 23, 35):
        one = check(x[i:i + 1], u[i:i + 1], t=t[i], k=k[i], p=p[i], m=m[i])
        assert one[0] == whole[i]


def test_settings_out_of_range_are_reported():
    x, u = noise(8, 500, "bf16")
    nan = float("nan")
    t = torch.tensor([1.0, -1.0, nan, INF, 1.0, 1.0, 1.0, 1.0]).cuda()
    p = torch.tensor([0.9, 0.9, 0.9, 0.9, nan, -0.1, 0.9, 0.9]).cuda()
    m = torch.tensor([0.0, 0.0, 0.0, 0.0, 0.0, 0.0, 1.5, nan]).cuda()
    (tok, lp, dlp, kept), err = run(x, u, temperature=t, top_p=p, min_p=m)
    assert err == 1
    assert tok[0] >= 0 and (tok[1:] == -1).all() and (lp[1:] == 0).all() and (kept[1:] == 0).all()
    uu = torch.tensor([-0.1, 1.0, nan, 0.5], dtype=torch.float64).cuda()
    (tok, _, _, _), err = run(x[:4], uu)
    assert err == 1 and (tok[:3] == -1).all() and tok[3] >= 0


def test_draws_follow_the_distribution():
    """One row drawn many times: the counts against the masses (chi-square, 99.99%)."""
    v, n = 50, 200_000
    g = torch.Generator("cuda").manual_seed(8)
    row = torch.randn(v, generator=g, device="cuda") * 1.5
    u = torch.rand(n, generator=g, device="cuda", dtype=torch.float64)
    tok = pkg.HeadSampler()(row.expand(n, v).contiguous(), u)[0]
    count = torch.bincount(tok, minlength=v).double()
    want = torch.softmax(row.double(), 0) * n
    chi = float(((count - want) ** 2 / want).sum())
    assert chi < 100.0  # 49 degrees of freedom: 100 is beyond the 99.99% point (94)


def test_same_answer_whatever_the_batch_and_stream():
    x, u = noise(700, 8200, "bf16", seed=21)
    sampler = pkg.HeadSampler()
    for f in ({}, dict(temperature=0.9, top_k=40, top_p=0.95), dict(top_p=0.9)):
        a = sampler(x, u, **f)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            b = sampler(x, u, **f)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        for i in (0, 133, 699):
            one = sampler(x[i:i + 1], u[i:i + 1], **f)
            assert all(torch.equal(p[i:i + 1], q) for p, q in zip(a, one))


def test_rows_past_two_to_the_31_elements():
    v = 65536
    n = (1 << 31) // v + 3
    big = torch.empty(n, v, dtype=torch.bfloat16, device="cuda")
    big[:n - 4] = 0
    x, u = noise(4, v, "bf16", seed=30)
    big[n - 4:] = x
    uu = torch.rand(n, dtype=torch.float64, device="cuda")
    uu[n - 4:] = u
    tok = pkg.HeadSampler()(big, uu)[0]
    want = pkg.HeadSampler()(x, u)[0]
    assert torch.equal(tok[n - 4:], want)
    assert torch.equal(tok[:n - 4], torch.floor(uu[:n - 4] * v).long())


def test_graph_capture():
    x, u = noise(9, 32000, "bf16", seed=2)
    sampler = pkg.HeadSampler()
    want = sampler(x, u, top_p=0.9)
    out = tuple(torch.zeros_like(o) for o in want)
    p = torch.full((9,), 0.9, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sampler(x, u, top_p=p, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, out))


def test_no_rows():
    x = torch.empty(0, 100, dtype=torch.bfloat16, device="cuda")
    out = pkg.HeadSampler()(x, torch.empty(0, dtype=torch.float64, device="cuda"))
    assert all(o.numel() == 0 for o in out)


def test_refusals():
    x, u = noise(4, 100, "bf16")
    sampler = pkg.HeadSampler()
    with pytest.raises(ValueError):
        sampler(x, u.float())
    with pytest.raises(ValueError):
        sampler(x, u[:3])
    with pytest.raises(ValueError):
        sampler(x.t(), u)
    with pytest.raises(ValueError):
        sampler(x, u, top_k=torch.ones(4, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        sampler(x, u, top_p=torch.ones(4))
    with pytest.raises(hlb.HeadlossError):
        sampler(x, None)
    with pytest.raises(hlb.HeadlossError):
        sampler(x.double(), u)
    with pytest.raises(hlb.HeadlossError):
        pkg.HeadSampler(softcap=-1.0)(x, u)
    with pytest.raises(hlb.HeadlossError):
        pkg.HeadSampler(logits_scale=0.0)(x, u)


# -------------------------------------------- rows that leave the ordinary way ----


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("sigma", [0.02, 0.5, 1.0])
def test_flat_rows(dtype, sigma):
    """Nearly uniform long rows: the cut's bin holds more tokens than can be ranked, in keys that
    differ and in keys that do not."""
    x, u = noise(3, 128_256, dtype, seed=11, sigma=sigma)
    for f in (dict(p=0.9), dict(t=0.7, p=0.5), dict(k=50_000, p=0.9), dict(k=70_000), dict(p=0.9, m=0.3),
              dict(k=100, p=0.95), {}):
        check(x, u, **f)


def test_long_rows_of_few_values():
    g = torch.Generator().manual_seed(17)
    x = torch.randint(-2, 3, (3, 151_936), generator=g).float() * 1.5
    u = torch.rand(3, generator=g, dtype=torch.float64)
    for dtype in (torch.bfloat16, torch.float32):
        for f in (dict(k=40), dict(k=60_000), dict(p=0.3), dict(p=0.9), dict(k=50_000, p=0.7),
                  dict(t=0.0), {}):
            check(x.to(dtype).cuda(), u.cuda(), **f)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("descending", [True, False])
def test_sorted_rows(dtype, descending):
    """A vocabulary in the order of its logits: all candidates lie in one part of the row."""
    x, u = noise(4, 128_256, dtype, seed=13)
    x = x.float().sort(dim=1, descending=descending).values.to(DT[dtype])
    for f in (dict(k=1), dict(k=20, p=0.9), dict(t=0.8, k=100, p=0.95), dict(k=128), dict(k=129), dict(p=0.95),
              dict(k=3000, p=0.9), {}):
        check(x, u, **f)


@pytest.mark.parametrize("v", [1000, 32_000, 151_936])
def test_one_token_has_it_all(v):
    """A peak 40 octaves above a flat body: every mass but its own rounds to nothing."""
    x = torch.full((3, v), -1.0)
    x[:, v // 3] = 30.0
    x[1, v - 1] = 30.0
    u = torch.tensor([0.0, 0.6, 0.999], dtype=torch.float64).cuda()
    for f in ({}, dict(p=0.9), dict(k=50, p=0.9), dict(k=5000), dict(m=0.5), dict(t=0.0)):
        tok = check(x.bfloat16().cuda(), u, **f)
        assert tok[0] == v // 3 and tok[2] == v // 3


def test_log_probs_do_not_depend_on_the_batch():
    """The model's log-probs are sums in fixed point: the same bits for a row alone and among
    others, although rows are then split over other numbers of CTAs."""
    x, u = noise(600, 32_000, "bf16", seed=41)
    sampler = pkg.HeadSampler()
    t = torch.full((600,), 0.8, device="cuda")
    p = torch.full((600,), 0.9, device="cuda")
    a = sampler(x, u, temperature=t, top_p=p)
    for i in (0, 311, 599):
        b = sampler(x[i:i + 1], u[i:i + 1], temperature=t[:1], top_p=p[:1])
        assert all(torch.equal(q[i:i + 1], r) for q, r in zip(a, b))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("offset", [1, 3, 7])
def test_views_off_the_grid(dtype, offset):
    """The base itself off the 16-byte grid: columns from `offset` on, as a view."""
    x, u = noise(5, 4000, dtype, seed=offset, pitch=4000 + offset)
    whole = torch.empty(5, 4000 + offset, dtype=DT[dtype], device="cuda")
    whole[:, :offset] = 100.0  # what lies before the view would win every draw
    whole[:, offset:] = x
    for f in ({}, dict(p=0.9), dict(t=0.8, k=40, p=0.9), dict(k=900)):
        check(whole[:, offset:], u, **f)
