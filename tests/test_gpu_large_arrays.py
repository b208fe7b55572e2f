"""Arrays past 2^31 elements: rows repeat with a short period, so every row has
to come out as the same row of a small call does, bit for bit."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
P = 4096  # rows of the period, a multiple of every tile
R = 4_300_000


@pytest.fixture(scope="module")
def moe():
    import combine_dispatch_amd as m
    m.lib()
    return m


def periodic(base):
    """base repeated along its first dimension to R rows."""
    return base.repeat(-(-R // base.shape[0]), *[1] * (base.dim() - 1))[:R].contiguous()


def same_rows(big, small):
    n = R // P * P
    for lo in range(0, n, 64 * P):
        part = big[lo:min(lo + 64 * P, n)]
        assert torch.equal(part.view(-1, *small.shape), small.expand(part.shape[0] // P, *small.shape))
    assert torch.equal(big[n:], small[:R - n])


def test_quantise_rows_and_product(moe):
    g = torch.Generator(DEV).manual_seed(1)
    K, N = 512, 24
    x = torch.randn(P, K, device=DEV, generator=g).bfloat16()
    w = torch.randn(1, N, K, device=DEV, generator=g)
    cw, sw = torch.empty(1, N, K, dtype=torch.uint8, device=DEV), torch.empty(1, 1, K // 128, device=DEV)
    moe.moe_quantise_weights(w, cw, sw)

    def run(x):
        n = x.shape[0]
        c, s = torch.empty(n, K, dtype=torch.uint8, device=DEV), torch.empty(K // 128, n, device=DEV)
        y = torch.empty(n, N, dtype=torch.bfloat16, device=DEV)
        moe.moe_quantise_rows(x, c, s)
        moe.moe_block_gemm(c, s, cw, sw, y)
        return c, s, y

    small, big = run(x), run(periodic(x))
    assert big[0].numel() > 2 ** 31
    same_rows(big[0], small[0])
    same_rows(big[1].t().contiguous(), small[1].t().contiguous())
    same_rows(big[2], small[2])


def test_quantise_columns_and_weight_gradient(moe):
    g = torch.Generator(DEV).manual_seed(2)
    C = 512
    x = torch.randn(P, C, device=DEV, generator=g).bfloat16()
    tail = 200
    off = torch.tensor([0, R // P * P, R // P * P + tail, R // P * P + tail], dtype=torch.int32, device=DEV)
    big = periodic(x)
    Rp = moe.moe_padded_rows(R, 3)
    c, s = torch.empty(C, Rp, dtype=torch.uint8, device=DEV), torch.empty(Rp // 128, C, dtype=torch.uint8, device=DEV)
    moe.moe_quantise_columns(big, c, s, offsets=off)
    assert c.numel() > 2 ** 31
    cs, ss = torch.empty(C, P, dtype=torch.uint8, device=DEV), torch.empty(P // 128, C, dtype=torch.uint8, device=DEV)
    moe.moe_quantise_columns(x, cs, ss)
    n = R // P
    for i in range(0, n, 64):
        m = min(64, n - i)
        assert torch.equal(c[:, i * P:(i + m) * P].reshape(C, m, P), cs[:, None].expand(C, m, P))
    assert torch.equal(s[:n * P // 128].view(n, P // 128, C), ss.expand(n, P // 128, C))
    # the second group's gradient is that of its 200 rows alone; the third is empty
    dw = torch.empty(3, C, C, dtype=torch.bfloat16, device=DEV)
    moe.moe_block_gemm_wgrad(c, s, c, s, dw, rows=R, offsets=off)
    ct, st = torch.empty(C, 256, dtype=torch.uint8, device=DEV), torch.empty(2, C, dtype=torch.uint8, device=DEV)
    moe.moe_quantise_columns(x[:tail].contiguous(), ct, st)
    one = torch.empty(1, C, C, dtype=torch.bfloat16, device=DEV)
    moe.moe_block_gemm_wgrad(ct, st, ct, st, one, rows=tail)
    assert torch.equal(dw[1], one[0]) and (dw[2] == 0).all() and torch.isfinite(dw[0]).all()


def test_gate_and_gradient(moe):
    g = torch.Generator(DEV).manual_seed(3)
    E, K, T = 512, 4, R
    l = torch.randn(P, E, device=DEV, generator=g).bfloat16()

    def run(l):
        n = l.shape[0]
        idx, w = torch.empty(n, K, dtype=torch.int64, device=DEV), torch.empty(n, K, device=DEV)
        moe.moe_gate(l, idx, w)
        d = torch.empty_like(l)
        moe.moe_gate_backward(l, d, topk_idx=idx, d_topk_w=w, opts=moe.gate_options())
        return idx, w, d

    small, big = run(l), run(periodic(l))
    assert big[2].numel() > 2 ** 31
    for b, s in zip(big, small):
        same_rows(b, s)
    # the balance loss of one long sequence: the counts of the period, times its number
    n = T // P * P
    loss, counts, slope = torch.empty(1, device=DEV), torch.empty(1, E, dtype=torch.int32, device=DEV), torch.empty(1, E, device=DEV)
    ws = torch.empty(moe.moe_balance_workspace_bytes(T, E, K), dtype=torch.uint8, device=DEV)
    moe.moe_balance_loss(periodic(l), big[0], 1.0, loss, counts, slope, ws,
                         seq_offsets=torch.tensor([0, n], dtype=torch.int32, device=DEV))
    assert torch.equal(counts[0].long(), torch.bincount(small[0].view(-1), minlength=E) * (T // P))
