"""The head's products in 8 bits against plain definitions in 64 bits.

Tolerance of a product, beside half a step of the output's type: the sum of a block's 128
products has at most 128 additions in the tensor core, each off by at most 2^-23 (a
truncation) of the magnitudes' sum, so 2^-16 of it; the product of the two scales and the KB scaled
additions round by 2^-24 each.  Codes and scales are exact."""
import math

import pytest
import torch

import gradient_row_online_gb300 as pkg
from gradient_row_online_gb300 import headloss as hl

pytestmark = pytest.mark.gpu

TOP = {"e4m3": 448.0, "e5m2": 57344.0}
TYPE = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
CODE = {"e4m3": hl.HEADLOSS_E4M3, "e5m2": hl.HEADLOSS_E5M2}


def quantised(x, kind, block):
    """The definition, block by block, on the CPU: codes (as the 8-bit type) and scales
    [ceil(rows / block)][ceil(cols / 128)]."""
    x = x.float().cpu()
    rows, cols = x.shape
    q = torch.empty(rows, cols, dtype=TYPE[kind])
    scales = torch.empty(-(-rows // block), -(-cols // 128))
    for j in range(scales.shape[1]):
        t = x[:, 128 * j:128 * j + 128]
        size = t.abs().amax(1)
        if block == 128:
            pad = torch.nn.functional.pad(size, (0, -rows % 128))
            size = pad.view(-1, 128).amax(1)
        s = torch.clamp(size * torch.tensor(1.0 / TOP[kind], dtype=torch.float32), min=2.0 ** -126)
        s = torch.where(torch.isfinite(size), s, math.nan)
        scales[:, j] = s
        inv = (1.0 / s).repeat_interleave(block)[:rows, None]
        q[:, 128 * j:128 * j + 128] = (t * inv).clamp(-TOP[kind], TOP[kind]).to(TYPE[kind])
    return q, scales


def values(q, scales, block):
    wide = scales.double().repeat_interleave(128, 1)[:, :q.shape[1]]
    return q.double() * wide.repeat_interleave(block, 0)[:q.shape[0]]


def run_quantise(x, kind, block, block_t):
    rows, cols = x.shape
    ldq, ldt = -(-cols // 16) * 16, -(-rows // 16) * 16
    q = torch.zeros(rows, ldq, dtype=torch.uint8, device="cuda")
    qt = torch.zeros(cols, ldt, dtype=torch.uint8, device="cuda")
    rb, cb = -(-rows // 128), -(-cols // 128)
    s = torch.zeros((cb, rows) if block == 1 else (rb, cb), device="cuda")
    st = torch.zeros((rb, cols) if block_t == 1 else (cb, rb), device="cuda")
    hl.headloss_fp8_quantize(x, rows, cols, x.stride(0), hl.dtype_code(x.dtype), CODE[kind], q, ldq, s, block,
                             qt, ldt, st, block_t)
    return (q[:, :cols].view(TYPE[kind]).cpu(), (s.t() if block == 1 else s).cpu(),
            qt[:, :rows].view(TYPE[kind]).cpu(), (st.t() if block_t == 1 else st).cpu())


def same_codes(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 130), (128, 128), (129, 257), (200, 77), (70, 1000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("kind,block,block_t", [("e4m3", 1, 128), ("e4m3", 128, 128), ("e5m2", 1, 1), ("e4m3", 128, 1)])
def test_codes_and_scales(rows, cols, dtype, kind, block, block_t):
    g = torch.Generator().manual_seed(rows * 1000 + cols)
    x = torch.randn(rows, cols, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))
    x[0, 0] = 0.0
    x = x.to(dtype)
    q, s, qt, st = run_quantise(x.cuda(), kind, block, block_t)
    rq, rs = quantised(x, kind, block)
    rqt, rst = quantised(x.t(), kind, block_t)
    assert torch.equal(s, rs) and torch.equal(st, rst)
    assert same_codes(q, rq) and same_codes(qt, rqt)


def test_codes_of_extreme_blocks():
    """Zeros, subnormals, the types' largest values, infinities and NaN, each in a block of its own."""
    x = torch.zeros(9, 256)
    x[1, :] = 1e-40
    x[2, 5] = 3e38
    x[3, 7], x[3, 130] = math.inf, 1.0
    x[4, 9] = math.nan
    x[5, 200] = -math.inf
    x[6, 0], x[6, 1] = 1e-38, -2e-41
    x[7, :] = 1e30 * torch.arange(256)
    q, s, qt, st = run_quantise(x.cuda(), "e4m3", 1, 1)
    rq, rs = quantised(x, "e4m3", 1)
    rqt, rst = quantised(x.t(), "e4m3", 1)
    assert torch.equal(s.nan_to_num(nan=-1.0), rs.nan_to_num(nan=-1.0))
    assert torch.equal(st.nan_to_num(nan=-1.0), rst.nan_to_num(nan=-1.0))
    for a, r, sc in ((q, rq, rs), (qt, rqt, rst)):
        fine = torch.isfinite(sc).repeat_interleave(128, 1)[:, :a.shape[1]]
        assert torch.equal(a.float()[fine], r.float()[fine])
    assert torch.isnan(rs[3, 0]) and rs[3, 1] == torch.tensor(1.0) * torch.tensor(1.0 / 448.0)
    assert torch.isnan(rs[4, 0]) and torch.isnan(rs[5, 1]) and not torch.isnan(rs[5, 0])


def random_codes(g, rows, cols, kind):
    """Every finite code, the small magnitudes as often as the large ones."""
    q = torch.randint(0, 256, (rows, cols), generator=g, dtype=torch.uint8)
    bad = ~torch.isfinite(q.view(TYPE[kind]).float())
    return torch.where(bad, torch.zeros_like(q), q)


def bound_of(dtype, ref, size, KB):
    return (torch.finfo(dtype).eps / 2 * ref.abs() + (2.0 ** -16 + (KB + 3) * 2.0 ** -24) * (1 + torch.finfo(dtype).eps) * size
            + torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps)


SIZES = [(1, 1, 1), (1, 128, 128), (2, 130, 4096), (3, 257, 130), (16, 1000, 1000), (17, 33, 2056), (32, 128, 700),
         (33, 513, 129), (64, 1000, 1024), (65, 300, 700), (100, 7, 3000), (128, 256, 128), (129, 257, 129),
         (200, 5003, 1000), (300, 100, 5003), (130, 1000, 16400), (1000, 2000, 256), (5003, 65, 7)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("out,at,bt,pad", [(torch.bfloat16, "e4m3", "e4m3", 0), (torch.float32, "e5m2", "e4m3", 3),
                                           (torch.float16, "e4m3", "e5m2", 8)])
def test_product(M, N, K, out, at, bt, pad):
    g = torch.Generator().manual_seed(M + 7 * N + 31 * K)
    KB, NB = -(-K // 128), -(-N // 128)
    ld = -(-K // 16) * 16 + 16
    a, b = random_codes(g, M, ld, at), random_codes(g, N, ld, bt)
    a[:, K:], b[:, K:] = 0x7f, 0x7f  # NaN in both types: past K nothing is read
    sa = torch.exp(torch.randn(M, KB, generator=g)) / TOP[at]
    sb = torch.exp(torch.randn(NB, KB, generator=g)) / TOP[bt]
    buf = torch.full((M, N + pad), 7.0, dtype=out, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    da, db, dsa, dsb = a.cuda(), b.cuda(), sa.t().contiguous().cuda(), sb.cuda()
    need = hl.headloss_fp8_workspace(M, N, K)
    work = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    for _ in range(2):
        hl.headloss_fp8_matmul(da, ld, dsa, CODE[at], db, ld, dsb, CODE[bt], M, N, K, buf, N + pad,
                               hl.dtype_code(out), work, need, err)
    got = buf.cpu()
    assert int(err) == 0
    assert (got[:, N:] == 7.0).all()
    va = values(a[:, :K].contiguous().view(TYPE[at]), sa, 1)
    vb = values(b[:, :K].contiguous().view(TYPE[bt]), sb, 128)
    ref, size = va @ vb.t(), va.abs() @ vb.abs().t()
    over = ref.abs() > torch.finfo(out).max
    off = (got[:, :N].double() - ref).abs()
    assert (off <= bound_of(out, ref, size, KB))[~over].all(), float((off / size)[~over].max())


@pytest.mark.parametrize("N,D,V", [(1, 256, 1000), (5, 200, 333), (70, 1000, 513), (200, 130, 2049)])
@pytest.mark.parametrize("dtype,master,grads", [(torch.bfloat16, torch.float32, "e4m3"),
                                                (torch.float32, torch.bfloat16, "e5m2"),
                                                (torch.float16, torch.float16, "e4m3")])
def test_head(N, D, V, dtype, master, grads):
    g = torch.Generator().manual_seed(N + D + V)
    w = (torch.randn(V, D, generator=g) * D ** -0.5).to(master)
    x = torch.randn(N, D, generator=g).to(dtype)
    dl = (torch.randn(N, V, generator=g) * 0.01).to(dtype)
    head = pkg.Fp8Head(w.cuda(), train=True, grads=grads)
    logits = head.logits(x.cuda())
    gh, gw = head.backward(dl.cuda(), x.cuda())
    assert logits.dtype == gh.dtype == dtype and gw.dtype == master and head.device_error() == 0
    vw = values(*quantised(w, "e4m3", 128), 128)
    for got, (qa, sa), vb in (
            (logits, quantised(x, "e4m3", 1), vw), (gh, quantised(dl, grads, 1), vw.t()),
            (gw, quantised(dl.t(), grads, 1), values(*quantised(x.t(), "e4m3", 128), 128))):
        va = values(qa, sa, 1)
        ref, size = va @ vb.t(), va.abs() @ vb.abs().t()
        off = (got.cpu().double() - ref).abs()
        assert (off <= bound_of(got.dtype, ref, size, sa.shape[1])).all()


def test_head_of_a_checkpoint_and_new_weights():
    g = torch.Generator().manual_seed(3)
    w = torch.randn(300, 200, generator=g)
    q, s = quantised(w, "e4m3", 128)
    held = pkg.Fp8Head.from_quantized(q.cuda(), s.cuda(), train=True)
    made = pkg.Fp8Head(w.cuda(), train=True)
    x, dl = torch.randn(9, 200, generator=g).cuda(), torch.randn(9, 300, generator=g).cuda()
    for a, b in ((held.logits(x), made.logits(x)), *zip(held.backward(dl, x, weight_dtype=torch.float32), made.backward(dl, x))):
        assert torch.equal(a, b)
    made.set_weight(2 * w.cuda())  # scales double, codes stay
    assert torch.equal(made.logits(x), 2 * held.logits(x))


def test_nonfinite_inputs_show():
    w = torch.randn(300, 256).cuda()
    head = pkg.Fp8Head(w, train=True)
    x = torch.randn(70, 256).cuda()
    x[3, 9] = math.inf
    bad = head.logits(x).isnan().any(1)
    assert bad[3] and int(bad.sum()) == 1
    w[200, 3] = math.nan
    head.set_weight(w)
    x[3, 9] = 0.0
    bad = head.logits(x[:2]).isnan().all(0)
    assert bad[128:256].all() and int(bad.sum()) == 128


def test_strided_inputs_outputs_and_empty():
    g = torch.Generator().manual_seed(5)
    w = torch.randn(300, 200, generator=g).cuda()
    head = pkg.Fp8Head(w, train=True)
    x, dl = torch.randn(40, 201, generator=g).cuda()[:, 1:], torch.randn(40, 333, generator=g).cuda()[:, :300]
    out = torch.full((40, 310), 5.0).cuda()
    got = head.logits(x, out=out[:, 3:303])
    assert torch.equal(got, head.logits(x.contiguous())) and (out[:, :3] == 5).all() and (out[:, 303:] == 5).all()
    a, b = head.backward(dl, x), head.backward(dl.contiguous(), x.contiguous())
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert head.logits(x[:0]).shape == (0, 300)
    gh, gw = head.backward(dl[:0], x[:0])
    assert gh.shape == (0, 200) and (gw == 0).all()


def test_rows_do_not_depend_on_their_neighbours():
    """A token alone and in a batch of the same kernel gives the same bits."""
    g = torch.Generator().manual_seed(6)
    head = pkg.Fp8Head(torch.randn(1000, 512, generator=g).cuda())
    x = torch.randn(16, 512, generator=g).bfloat16().cuda()
    assert torch.equal(head.logits(x)[5:6], head.logits(x[5:6]))


def test_captured_and_replayed():
    g = torch.Generator().manual_seed(7)
    head = pkg.Fp8Head(torch.randn(1000, 512, generator=g).cuda(), train=True)
    x, dl = torch.randn(70, 512, generator=g).cuda(), torch.randn(70, 1000, generator=g).cuda()
    want = [head.logits(x), *head.backward(dl, x)]
    keep = x.clone(), dl.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = [head.logits(x), *head.backward(dl, x)]
    x.zero_(), dl.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all((t == 0).all() for t in got)
    x.copy_(keep[0]), dl.copy_(keep[1])
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("N", [1, 7, 64, 130, 392])
@pytest.mark.parametrize("extra", [0, 1, 8])
def test_out_that_starts_anywhere(dtype, N, extra):
    """The bits do not depend on where rows of out start, and what lies beside them stays."""
    g = torch.Generator().manual_seed(N)
    head = pkg.Fp8Head(torch.randn(N, 200, generator=g).cuda())
    x = torch.randn(37, 200, generator=g).to(dtype).cuda()
    want = head.logits(x)
    for o in range(8):
        buf = torch.full((39, N + 8 + extra), 7.0, dtype=dtype, device="cuda")
        assert torch.equal(head.logits(x, out=buf[1:38, o:o + N]), want)
        buf[1:38, o:o + N] = 7.0
        assert (buf == 7.0).all()


@pytest.mark.parametrize("M,N,K", [(1, 1000, 256), (3, 257, 130), (70, 513, 1000), (200, 2049, 77), (1, 4096, 32000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_is_the_two_calls(M, N, K, dtype):
    g = torch.Generator().manual_seed(M + N + K)
    x = torch.randn(M, K, generator=g).to(dtype).cuda()
    code, ld = hl.dtype_code(dtype), -(-K // 16) * 16
    bq, bs, _, _ = run_quantise(torch.randn(N, K, generator=g).cuda(), "e4m3", 128, 128)
    b = torch.zeros(N, ld, dtype=torch.uint8)
    b[:, :K] = bq.view(torch.uint8)
    b, bs = b.cuda(), bs.cuda()
    a, sa = torch.empty(M, ld, dtype=torch.uint8, device="cuda"), torch.empty(-(-K // 128), M, device="cuda")
    out = torch.empty(2, M, N, dtype=dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    hl.headloss_fp8_quantize(x, M, K, K, code, CODE["e4m3"], a, ld, sa, 1, None, 0, None, 0)
    need = hl.headloss_fp8_workspace(M, N, K)
    work = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    hl.headloss_fp8_matmul(a, ld, sa, CODE["e4m3"], b, ld, bs, CODE["e4m3"], M, N, K, out[0], N, code, work, need, err)
    need = hl.headloss_fp8_linear_workspace(M, N, K)
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    hl.headloss_fp8_linear(x, K, code, b, ld, bs, CODE["e4m3"], M, N, K, out[1], N, code, work, need, err)
    assert int(err) == 0 and torch.equal(out[0], out[1])
