"""The head's products in 8 bits on matrices whose elements pass 32 bits: a long batch's logits and gradient."""
import pytest
import torch

import gradient_row_online_gb300 as pkg
from gradient_row_online_gb300 import headloss as hl
from tests.test_fp8_gpu import CODE, TYPE, bound_of, values

pytestmark = pytest.mark.gpu

ROWS, V = 33793, 128256  # 4.3e9 elements
assert ROWS * V > 1 << 32


def test_logits_of_a_long_batch():
    g = torch.Generator("cuda").manual_seed(1)
    head = pkg.Fp8Head(torch.randn(V, 200, generator=g, device="cuda"))
    x = torch.randn(ROWS, 200, generator=g, device="cuda").bfloat16()
    out = head.logits(x)
    assert torch.equal(out[-131:], head.logits(x[-131:])) and torch.equal(out[:131], head.logits(x[:131]))
    # rows that start anywhere are not stored by the tensor map
    buf = torch.empty(ROWS * (V + 1), dtype=torch.bfloat16, device="cuda").view(ROWS, V + 1)
    assert torch.equal(head.logits(x, out=buf[:, :V])[-131:], out[-131:]) and head.device_error() == 0


def test_codes_of_a_long_gradient():
    g = torch.Generator("cuda").manual_seed(2)
    x = torch.empty(ROWS, V, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    ldt = -(-ROWS // 16) * 16
    q, qt = torch.empty(ROWS, V, dtype=torch.uint8, device="cuda"), torch.empty(V, ldt, dtype=torch.uint8, device="cuda")
    kb, rb = -(-V // 128), -(-ROWS // 128)
    s, st = torch.empty(kb, ROWS, device="cuda"), torch.empty(rb, V, device="cuda")
    hl.headloss_fp8_quantize(x, ROWS, V, V, hl.HEADLOSS_BF16, CODE["e4m3"], q, V, s, 1, qt, ldt, st, 1)
    first = ROWS // 128 * 128 - 128  # the last two rows of tiles by themselves
    part, n = x[first:], ROWS - first
    ld = -(-n // 16) * 16
    pq, pt = torch.empty(n, V, dtype=torch.uint8, device="cuda"), torch.empty(V, ld, dtype=torch.uint8, device="cuda")
    ps, pst = torch.empty(kb, n, device="cuda"), torch.empty(2, V, device="cuda")
    hl.headloss_fp8_quantize(part, n, V, V, hl.HEADLOSS_BF16, CODE["e4m3"], pq, V, ps, 1, pt, ld, pst, 1)
    assert torch.equal(q[first:], pq) and torch.equal(s[:, first:], ps)
    assert torch.equal(qt[:, first:ROWS], pt[:, :n]) and torch.equal(st[-2:], pst)
    # grad_hidden of the whole, its last rows against 64 bits
    N, err = 256, torch.zeros(1, dtype=torch.int32, device="cuda")
    b = (torch.randint(0, 100, (N, V), generator=g, device="cuda") + 10).to(torch.uint8)
    sb = torch.rand(2, kb, generator=g, device="cuda") / 448
    out = torch.empty(ROWS, N, device="cuda")
    need = hl.headloss_fp8_workspace(ROWS, N, V)
    work = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    hl.headloss_fp8_matmul(q, V, s, CODE["e4m3"], b, V, sb, CODE["e4m3"], ROWS, N, V, out, N, hl.HEADLOSS_FP32, work, need, err)
    rows = [0, 1, ROWS // 2, ROWS - 2, ROWS - 1]
    va = values(q[rows].view(TYPE["e4m3"]), s.t()[rows], 1)
    vb = values(b.view(TYPE["e4m3"]), sb, 128)
    ref, size = va @ vb.t(), va.abs() @ vb.abs().t()
    assert int(err) == 0 and ((out[rows].double() - ref).abs() <= bound_of(torch.float32, ref, size, kb)).all()
