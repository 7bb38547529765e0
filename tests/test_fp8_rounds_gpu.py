"""The head's product in 8 bits where a CTA has several tiles one after the other: rounds of tiles, a last round that is
not full, whole or with its K in parts, in every output type and alignment, against 64 bits. Tolerance as in test_fp8_gpu."""
import pytest
import torch

from gradient_row_online_gb300 import headloss as hl
from tests.test_fp8_gpu import CODE, TOP, TYPE, bound_of, values

pytestmark = pytest.mark.gpu


def codes(g, rows, ld, kind):
    q = torch.randint(0, 256, (rows, ld), generator=g, dtype=torch.uint8, device="cuda")
    return torch.where(torch.isfinite(q.view(TYPE[kind]).float()), q, 0).to(torch.uint8)


def columns(M, rounds, more):
    """Columns whose tiles of 128 x 256 fill every SM `rounds` times, and `more` column tiles."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    tall = -(-M // 128)
    return 256 * (-(-rounds * sms // tall) + more)


@pytest.mark.parametrize("M", [1, 37, 64, 65, 200, 300])
@pytest.mark.parametrize("K,parts", [(100, False), (1100, False), (5243, True)])  # 1, 9 and 41 blocks: odd numbers of them
@pytest.mark.parametrize("out,at,bt,short,pad,off", [(torch.bfloat16, "e4m3", "e4m3", 0, 0, 0), (torch.float32, "e5m2", "e4m3", 100, 3, 1),
                                                     (torch.float16, "e4m3", "e5m2", 5, 8, 3)])
def test_rounds_of_tiles(M, K, parts, out, at, bt, short, pad, off):
    g = torch.Generator("cuda").manual_seed(M + K)
    N = columns(M, 2, 3) - short
    KB, NB, ld = -(-K // 128), -(-N // 128), -(-K // 16) * 16
    a, b = codes(g, M, ld, at), codes(g, N, ld, bt)
    a[:, K:], b[:, K:] = 0x7f, 0x7f
    sa = torch.exp(torch.randn(M, KB, generator=g, device="cuda")) / TOP[at]
    sb = torch.exp(torch.randn(NB, KB, generator=g, device="cuda")) / TOP[bt]
    buf = torch.full((M + 1, N + pad), 7.0, dtype=out, device="cuda")
    got = buf.view(-1)[off:off + M * (N + pad)].view(M, N + pad)  # (rows that start `off` elements on)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    need = hl.headloss_fp8_workspace(M, N, K)
    assert (need > 0) == parts
    work = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    turned = sa.t().contiguous()
    for _ in range(2):
        hl.headloss_fp8_matmul(a, ld, turned, CODE[at], b, ld, sb, CODE[bt], M, N, K, got, N + pad, hl.dtype_code(out), work,
                               need, err)
    assert int(err) == 0
    assert (got[:, N:] == 7.0).all() and (buf.view(-1)[:off] == 7.0).all() and (buf.view(-1)[off + M * (N + pad):] == 7.0).all()
    va = values(a[:, :K].contiguous().view(TYPE[at]), sa, 1)
    over = 0
    for j in range(0, N, 1 << 15):  # 256 blocks of scales at a time
        n = min(N, j + (1 << 15))
        vb = values(b[j:n, :K].contiguous().view(TYPE[bt]), sb[j // 128:-(-n // 128)], 128)
        ref, size = va @ vb.t(), va.abs() @ vb.abs().t()
        fine = ref.abs() <= torch.finfo(out).max
        off_by = (got[:, j:n].double() - ref).abs()
        assert (off_by <= bound_of(out, ref, size, KB))[fine].all(), float((off_by / size)[fine].max())
        over += int((~fine).sum())
    assert over < M * N // 100


@pytest.mark.parametrize("M", [1, 48, 130])
@pytest.mark.parametrize("K", [300, 1100, 5243])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_over_rounds_is_the_two_calls(M, K, dtype):
    g = torch.Generator("cuda").manual_seed(M + K)
    N, KB, ld, code = columns(M, 2, 2) - 3, -(-K // 128), -(-K // 16) * 16, hl.dtype_code(dtype)
    x = torch.randn(M, K, generator=g, device="cuda").to(dtype)
    b, sb = codes(g, N, ld, "e4m3"), torch.rand(-(-N // 128), KB, generator=g, device="cuda") / 448
    a, sa = torch.empty(M, ld, dtype=torch.uint8, device="cuda"), torch.empty(KB, M, device="cuda")
    out = torch.zeros(2, M, N, dtype=dtype, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    need, all_need = hl.headloss_fp8_workspace(M, N, K), hl.headloss_fp8_linear_workspace(M, N, K)
    work = torch.empty(all_need, dtype=torch.uint8, device="cuda")
    hl.headloss_fp8_quantize(x, M, K, K, code, CODE["e4m3"], a, ld, sa, 1, None, 0, None, 0)
    hl.headloss_fp8_matmul(a, ld, sa, CODE["e4m3"], b, ld, sb, CODE["e4m3"], M, N, K, out[0], N, code, work, need, err)
    for _ in range(3):
        out[1].zero_()
        hl.headloss_fp8_linear(x, K, code, b, ld, sb, CODE["e4m3"], M, N, K, out[1], N, code, work, all_need, err)
        assert int(err) == 0 and torch.equal(out[0], out[1])
    assert out[0].isfinite().all() and out[0].count_nonzero() > M * N * 9 // 10
