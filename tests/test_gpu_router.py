"""GPU tests of the router (include/moe_gate.h) against float64 forms of its
formulas, computed on the CPU.

Tolerances, in u = 2^-24 (half a step of float32, relative).  D = the largest
difference of two logits of a row.  One score exp(l - top) is off by
(D + 4) u: the difference is rounded once (D u in the exponent) and expf errs
by at most 2 steps.  1 / (1 + exp(-l)) errs by no more than 10 u.  A sum of n
positive terms adds n u.  So a normalised score errs by
eps = (2 (D + 4) + n + 16) u relative, n the number of terms.  A gradient
q (g - sum g q) errs by at most 4 eps of q (max |g| + |sum g q|); where 1 - s
enters it is off by another 16 u absolute.  bf16 results add half a step, 2^-8.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U = 2.0 ** -24


@pytest.fixture(scope="module")
def moe():
    import combine_dispatch_amd as m
    m.lib()
    return m


def make_logits(T, E, dtype, seed, std=1.5):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn(T, E, generator=g) * std + 0.5 * torch.randn(1, E, generator=g)
    return l.to(dtype)


def softmax64(l):
    m = l.amax(1, keepdim=True)
    z = torch.exp(l - torch.where(torch.isinf(m) & (m < 0), torch.zeros_like(m), m))
    s = z.sum(1, keepdim=True)
    return torch.where(s == 0, torch.zeros_like(z), z / s)


def sigmoid64(l):
    return 1 / (1 + torch.exp(-l))


def ref_gate(l, K, score, renorm, scale, bias=None, mask=None):
    """(idx, w) in float64 by full sorts; ties to the lower index, -inf never chosen."""
    l = l.double()
    s = softmax64(l) if score == "softmax" else sigmoid64(l)
    key = l.clone() if bias is None else sigmoid64(l) + bias.double()
    key[torch.isinf(l) & (l < 0)] = -np.inf
    val, idx = torch.sort(key, dim=1, descending=True, stable=True)
    val, idx = val[:, :K], idx[:, :K].clone()
    sel = s.gather(1, idx)
    none = torch.isinf(val) & (val < 0)
    if mask is not None:
        none |= (mask == 0)[:, None]
    sel = torch.where(none, torch.zeros_like(sel), sel)
    w = sel
    if renorm:
        t = sel.sum(1, keepdim=True)
        w = torch.where(t == 0, torch.zeros_like(sel), sel / t)
    idx[none] = -1
    return idx, scale * w


def spread(l):
    f = l.double()
    f = f[torch.isfinite(f)]
    return float(f.max() - f.min()) if f.numel() else 0.0


def run_gate(moe, l, K, score, renorm, scale=1.0, bias=None, mask=None):
    T = l.shape[0]
    idx = torch.full((T, K), -7, dtype=torch.int64, device=DEV)
    w = torch.full((T, K), 7.0, device=DEV)
    moe.moe_gate(l.to(DEV), idx, w, bias=None if bias is None else bias.to(DEV),
                 token_mask=None if mask is None else mask.to(DEV),
                 opts=moe.gate_options(score=score, renormalise=renorm, scale=scale))
    return idx.cpu(), w.cpu()


SIZES = [(1, 1, 1), (3, 2, 2), (17, 7, 3), (16, 8, 2), (33, 16, 16), (5, 17, 4), (257, 32, 8), (20, 33, 5),
         (64, 64, 6), (31, 100, 9), (130, 128, 8), (64, 256, 8), (9, 300, 12), (10, 513, 17), (7, 1024, 64)]


@pytest.mark.parametrize("T,E,K", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("mode", ["softmax", "softmax_raw", "sigmoid", "sigmoid_raw", "sigmoid_bias"])
def test_gate(moe, T, E, K, dtype, mode):
    l = make_logits(T, E, dtype, seed=T * 1000 + E)
    score, renorm = mode.split("_")[0], not mode.endswith("raw")
    g = torch.Generator().manual_seed(5)
    bias = 0.1 * torch.randn(E, generator=g) if mode.endswith("bias") else None
    mask = (torch.rand(T, generator=g) < 0.8).to(torch.uint8) if T > 4 else None
    idx, w = run_gate(moe, l, K, score, renorm, 2.5, bias, mask)
    ridx, rw = ref_gate(l, K, score, renorm, 2.5, bias, mask)
    assert torch.equal(idx, ridx)
    eps = (2 * (spread(l) + 4) + E + 16) * U
    assert ((w.double() - rw).abs() <= eps * rw.abs()).all(), float(((w - rw).abs() / rw.abs()).nan_to_num().max())


def test_gate_ties_go_to_the_lower_index(moe):
    l = torch.zeros(5, 96)
    l[1] = torch.arange(96) % 3
    l[2, 10:20] = -0.0  # equal to +0
    l[3] = torch.finfo(torch.float32).min  # the lowest value is an ordinary logit
    l[4, 90] = 1.0
    for score in ("softmax", "sigmoid"):
        idx, w = run_gate(moe, l, 6, score, True)
        ridx, rw = ref_gate(l, 6, score, True, 1.0)
        assert torch.equal(idx, ridx)
        if score == "softmax":
            # of the lowest values alone: an even softmax of the chosen ones
            assert torch.allclose(w[3], torch.full((6,), 1 / 6), atol=2 * U)
    # all keys equal with a bias as well: the float64 choice
    idx, _ = run_gate(moe, torch.zeros(3, 96), 6, "sigmoid", True, bias=torch.zeros(96))
    assert torch.equal(idx, torch.arange(6).expand(3, 6))


def test_gate_keys_closer_than_float32(moe):
    """Biases that make the keys of row 0 meet within a step of float32: the
    choice has to be that of float64 keys."""
    for E, K in ((24, 8), (64, 16), (256, 8), (700, 33)):
        l = make_logits(40, E, torch.float32, seed=E)
        bias = (0.75 - sigmoid64(l[0].double())).float()
        ridx, _ = ref_gate(l, K, "sigmoid", True, 1.0, bias)
        f32 = torch.sort(torch.sigmoid(l[0]) + bias, descending=True, stable=True)[1][:K]
        idx, w = run_gate(moe, l, K, "sigmoid", True, bias=bias)
        assert torch.equal(idx, ridx)
        assert not torch.equal(f32, ridx[0])  # float32 keys would not do


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_gate_rows_with_few_or_no_experts(moe, score, renorm):
    l = make_logits(6, 40, torch.float32, seed=3)
    l[0] = -np.inf
    l[1, 2:] = -np.inf
    l[2, :39] = -np.inf
    bias = torch.zeros(40)
    bias[0] = -np.inf  # a bias of -inf takes the expert out as well
    for b in ([None, bias] if score == "sigmoid" else [None]):
        idx, w = run_gate(moe, l, 4, score, renorm, bias=b)
        ridx, rw = ref_gate(l, 4, score, renorm, 1.0, b)
        assert torch.equal(idx, ridx)
        assert torch.isfinite(w).all()
        assert ((w.double() - rw).abs() <= (2 * (spread(l) + 4) + 56) * U * rw).all()
        assert (idx[0] == -1).all() and (w[0] == 0).all()


def test_gate_nan_and_inf(moe):
    l = make_logits(3, 32, torch.float32, seed=4)
    l[0, 9] = float("nan")
    l[1, 5] = float("inf")
    idx, w = run_gate(moe, l, 3, "softmax", True)
    assert idx[0, 0] == 9 and torch.isnan(w[0]).all()  # NaN reaches the weights
    assert idx[1, 0] == 5 and torch.isnan(w[1]).any()  # inf - inf, as softmax has it
    assert torch.isfinite(w[2]).all()
    idx, w = run_gate(moe, l, 3, "sigmoid", False)
    assert idx[0, 0] == 9 and torch.isnan(w[0, 0]) and torch.isfinite(w[0, 1:]).all()
    assert idx[1, 0] == 5 and w[1, 0] == 1.0
    # a masked token's NaN stays out
    idx, w = run_gate(moe, l, 3, "softmax", True, mask=torch.tensor([0, 0, 1], dtype=torch.uint8))
    assert (idx[:2] == -1).all() and (w[:2] == 0).all()


def test_gate_unaligned_rows(moe):
    """A logits view that starts off a 16-byte boundary takes the narrow loads."""
    for dtype in (torch.float32, torch.bfloat16):
        base = make_logits(1, 1 + 20 * 64, dtype, seed=8).to(DEV).view(-1)
        l = base[1:].view(20, 64)
        idx = torch.empty(20, 4, dtype=torch.int64, device=DEV)
        w = torch.empty(20, 4, device=DEV)
        moe.moe_gate(l, idx, w)
        ridx, rw = ref_gate(l.cpu(), 4, "softmax", True, 1.0)
        assert torch.equal(idx.cpu(), ridx)


def ref_grad(l, idx, dw, score, renorm, scale, slope=None, d_loss=None, seq=None, mask=None):
    """The gradient's formulas in float64, and the magnitude its error scales with."""
    l = l.double()
    T, E = l.shape
    soft = score == "softmax"
    s = softmax64(l) if soft else sigmoid64(l)
    d, mag = torch.zeros_like(l), torch.zeros_like(l)
    if idx is not None:
        ok = (idx >= 0) & (idx < E)
        at = torch.where(ok, idx, 0)
        g = torch.where(ok, scale * dw.double(), torch.zeros(()).double())
        sel = torch.where(ok, s.gather(1, at), torch.zeros(()).double())
        tot = sel.sum(1, keepdim=True)
        q = torch.where(tot == 0, torch.zeros_like(sel), sel / tot) if renorm else sel
        dot = (g * q).sum(1, keepdim=True)
        G = g.abs().amax(1, keepdim=True)
        if soft and not renorm:
            full = torch.zeros_like(l).scatter_add(1, at, g)
            d = s * (full - dot)
            mag = s * (full.abs() + G)
        else:
            term = q * (g - dot) if renorm else g * sel
            d = d.scatter_add(1, at, term * (1 if soft else 1 - sel))
            mag = mag.scatter_add(1, at, q * 2 * G)
    if slope is not None:
        p = s / s.sum(1, keepdim=True)
        f = torch.zeros_like(l)
        for q_, (a, b) in enumerate(zip(seq, seq[1:])):
            f[a:b] = slope[q_].double() * d_loss
        dot = (f * p).sum(1, keepdim=True)
        d = d + p * (f - dot) * (1 if soft else 1 - s)
        mag = mag + p * (f.abs() + f.abs().amax(1, keepdim=True))
    if mask is not None:
        d = d * (mask != 0)[:, None]
    return d, mag


def check_grad(got, ref, mag, l, E):
    eps = (2 * (spread(l) + 4) + E + 16) * U
    tol = (4 * eps + 32 * U) * mag + (2.0 ** -8 if got.dtype == torch.bfloat16 else U) * ref.abs()
    bad = (got.double() - ref).abs() > tol
    assert not bad.any(), float(((got.double() - ref).abs() / tol.clamp_min(1e-300)).max())


@pytest.mark.parametrize("T,E,K", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("mode", ["softmax", "softmax_raw", "sigmoid", "sigmoid_raw"])
@pytest.mark.parametrize("parts", ["gate", "balance", "both"])
def test_gradient(moe, T, E, K, dtype, mode, parts):
    l = make_logits(T, E, dtype, seed=T + E)
    score, renorm = mode.split("_")[0], not mode.endswith("raw")
    g = torch.Generator().manual_seed(6)
    mask = (torch.rand(T, generator=g) < 0.8).to(torch.uint8) if T % 2 else None
    idx, dw, slope, d_loss, seq = None, None, None, None, None
    o = moe.gate_options(score=score, renormalise=renorm, scale=1.5)
    kw = {}
    if parts != "balance":
        idx, _ = ref_gate(l, K, score, renorm, 1.5, None, mask)
        if K > 1:
            idx[::3, K - 1] = -1  # a masked slot
        dw = torch.randn(T, K, generator=g)
        kw.update(topk_idx=idx.to(DEV), d_topk_w=dw.to(DEV))
    if parts != "gate":
        cuts = sorted(torch.randint(0, T + 1, (4,), generator=g).tolist())
        seq = [0, *cuts, T] if T > 1 else [0, 1]
        slope = torch.rand(len(seq) - 1, E, generator=g)
        d_loss = 0.7
        kw.update(slope=slope.to(DEV), d_loss=torch.tensor([d_loss], device=DEV),
                  seq_offsets=torch.tensor(seq, dtype=torch.int32, device=DEV))
    d = torch.full((T, E), 9.0, dtype=dtype, device=DEV)
    moe.moe_gate_backward(l.to(DEV), d, token_mask=None if mask is None else mask.to(DEV), opts=o, **kw)
    ref, mag = ref_grad(l, idx, dw, score, renorm, 1.5, slope, np.float32(d_loss or 0), seq, mask)
    check_grad(d.cpu(), ref, mag, l, E)


@pytest.mark.parametrize("mode", ["softmax", "softmax_raw", "sigmoid", "sigmoid_raw"])
def test_gradient_against_differences(moe, mode):
    """Central differences of the float64 gate with the choice held fixed.
    Their own error is h^2 / 6 times the third derivative (below 4 max|dw|):
    h = 1e-4 leaves 1e-8, far under the kernel's float32 error bound."""
    score, renorm = mode.split("_")[0], not mode.endswith("raw")
    T, E, K, h = 6, 12, 4, 1e-4
    l = make_logits(T, E, torch.float32, seed=2)
    idx, _ = ref_gate(l, K, score, renorm, 1.0)
    dw = torch.randn(T, K, generator=torch.Generator().manual_seed(1))

    def value(x):
        s = softmax64(x) if score == "softmax" else sigmoid64(x)
        sel = s.gather(1, idx)
        w = sel / sel.sum(1, keepdim=True) if renorm else sel
        return (w * dw.double()).sum(1)

    d = torch.empty(T, E, device=DEV)
    moe.moe_gate_backward(l.to(DEV), d, topk_idx=idx.to(DEV), d_topk_w=dw.to(DEV),
                          opts=moe.gate_options(score=score, renormalise=renorm))
    for e in range(E):
        x = l.double()
        step = torch.zeros_like(x)
        step[:, e] = h
        fd = (value(x + step) - value(x - step)) / (2 * h)
        assert (d[:, e].cpu().double() - fd).abs().max() <= 1e-8 + 4 * (2 * (spread(l) + 4) + E + 48) * U * 2 * float(dw.abs().max())


def test_gradient_ignores_slots_and_tokens_outside(moe):
    T, E, K = 9, 32, 2
    l = make_logits(T, E, torch.float32, seed=1)
    idx = torch.tensor([[-1, -5], [E, 3], [1 << 40, -(1 << 40)]] + [[0, 1]] * 6)
    dw = torch.randn(T, K, generator=torch.Generator().manual_seed(1))
    d = torch.full((T, E), 9.0, device=DEV)
    moe.moe_gate_backward(l.to(DEV), d, topk_idx=idx.to(DEV), d_topk_w=dw.to(DEV))
    ref, mag = ref_grad(l, idx, dw, "softmax", True, 1.0)
    check_grad(d.cpu(), ref, mag, l, E)
    assert (d[0] == 0).all() and (d[2] == 0).all()
    # tokens before the first and behind the last sequence have no balance part
    slope = torch.ones(1, E, device=DEV) * torch.arange(E, device=DEV)
    moe.moe_gate_backward(l.to(DEV), d, slope=slope, d_loss=torch.ones(1, device=DEV),
                          seq_offsets=torch.tensor([2, 7], dtype=torch.int32, device=DEV))
    assert (d[:2] == 0).all() and (d[7:] == 0).all() and (d[2:7] != 0).any(1).all()


def ref_balance(l, idx, seq, coef, score, mask):
    l = l.double()
    T, E = l.shape
    s = softmax64(l) if score == "softmax" else sigmoid64(l)
    t = s.sum(1, keepdim=True)
    p = torch.where(t == 0, torch.zeros_like(s), s / t)
    live = torch.ones(T, dtype=torch.bool) if mask is None else mask != 0
    S = len(seq) - 1
    counts = torch.zeros(S, E, dtype=torch.int32)
    slope = torch.zeros(S, E, dtype=torch.float64)
    loss = 0.0
    n = [int(live[a:b].sum()) for a, b in zip(seq, seq[1:])]
    used = sum(v > 0 for v in n)
    for q, (a, b) in enumerate(zip(seq, seq[1:])):
        hit = idx[a:b][live[a:b]].reshape(-1)
        hit = hit[(hit >= 0) & (hit < E)]
        counts[q] = torch.bincount(hit, minlength=E).int()
        if n[q] and hit.numel():
            slope[q] = coef * E * counts[q].double() / (hit.numel() * n[q] * used)
            loss += float((slope[q] * p[a:b][live[a:b]].sum(0)).sum())
    return loss, counts, slope


def run_balance(moe, l, idx, seq, coef, score, mask=None):
    T, E = l.shape
    S = len(seq) - 1 if seq is not None else 1
    loss = torch.full((1,), 7.0, device=DEV)
    counts = torch.full((S, E), 7, dtype=torch.int32, device=DEV)
    slope = torch.full((S, E), 7.0, device=DEV)
    ws = torch.full((moe.moe_balance_workspace_bytes(T, E, idx.shape[1], S),), 0xA5, dtype=torch.uint8, device=DEV)
    moe.moe_balance_loss(l.to(DEV), idx.to(DEV), coef, loss, counts, slope, ws,
                         seq_offsets=None if seq is None else torch.tensor(seq, dtype=torch.int32, device=DEV),
                         token_mask=None if mask is None else mask.to(DEV), opts=moe.gate_options(score=score))
    return loss.cpu(), counts.cpu(), slope.cpu()


def check_balance(got, ref, l, E):
    eps = (2 * (spread(l) + 4) + E + 32) * U
    assert torch.equal(got[1], ref[1])
    assert ((got[2].double() - ref[2]).abs() <= 2 * U * ref[2]).all()
    assert abs(float(got[0]) - ref[0]) <= eps * ref[0]


BALANCE = [  # T, E, K, sequence offsets
    (1, 1, 1, None), (7, 5, 2, [0, 0, 3, 3, 7, 7]), (31, 16, 4, None), (32, 32, 8, [0, 32]),
    (33, 33, 2, [0, 32, 33]), (64, 100, 3, [0, 1, 2, 33, 34, 64]), (509, 32, 8, None), (700, 130, 6, [0, 96, 96, 320, 700]),
    (1000, 256, 8, [0] * 300 + [500] * 200 + [1000]), (65, 1024, 64, [5, 40, 60]), (4099, 8, 2, [0, 4099]),
    (300, 600, 1, list(range(301)))]


@pytest.mark.parametrize("T,E,K,seq", BALANCE)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_balance_loss(moe, T, E, K, seq, dtype, score):
    l = make_logits(T, E, dtype, seed=T + E)
    mask = (torch.rand(T, generator=torch.Generator().manual_seed(3)) < 0.7).to(torch.uint8) if T % 2 else None
    idx = torch.argsort(l.float(), dim=1, descending=True)[:, :K].contiguous()
    idx[::5, 0] = -1
    idx[1::7, K - 1] = E  # out of range: not counted
    ref = ref_balance(l, idx, seq or [0, T], 0.01, score, mask)
    check_balance(run_balance(moe, l, idx, seq, 0.01, score, mask), ref, l, E)


def test_balance_degenerate(moe):
    E = 24
    l = make_logits(50, E, torch.float32, seed=1)
    l[7] = -np.inf  # a token without experts: probability 0 everywhere, still a token
    idx = torch.randint(0, E, (50, 3), generator=torch.Generator().manual_seed(1))
    # a sequence of padding only, and one without counted slots
    mask = torch.ones(50, dtype=torch.uint8)
    mask[10:20] = 0
    idx[30:40] = -1
    seq = [0, 10, 20, 30, 40, 50]
    for score in ("softmax", "sigmoid"):
        check_balance(run_balance(moe, l, idx, seq, 1.0, score, mask), ref_balance(l, idx, seq, 1.0, score, mask), l, E)
    loss, counts, slope = run_balance(moe, l, idx, seq, 1.0, "softmax", torch.zeros(50, dtype=torch.uint8))
    assert float(loss) == 0 and (counts == 0).all() and (slope == 0).all()
    # no tokens at all
    loss, counts, slope = run_balance(moe, l[:0], idx[:0], None, 1.0, "softmax")
    assert float(loss) == 0 and (counts == 0).all() and (slope == 0).all()
    # an even router has loss = coef
    even = torch.zeros(64, 16)
    idx = (torch.arange(64 * 4) % 16).view(64, 4)
    loss, counts, slope = run_balance(moe, even, idx, None, 0.5, "softmax")
    assert abs(float(loss) - 0.5) <= 64 * U and (counts == 16).all()


def test_balance_bad_offsets_stay_in_bounds(moe):
    """Out of order and out of range: some result, finite, nothing written past the outputs."""
    l = make_logits(100, 8, torch.float32, seed=1)
    idx = torch.randint(0, 8, (100, 2), generator=torch.Generator().manual_seed(1))
    S = 4
    for seq in ([0, 90, 10, 300, 50], [-5, 20, 10, 1 << 30, 100], [100, 0, 0, 0, -(1 << 31)]):
        pad = torch.full((S + 2, 8), 7, dtype=torch.int32, device=DEV)
        slope = torch.full((S + 2, 8), 7.0, device=DEV)
        loss = torch.zeros(1, device=DEV)
        ws = torch.zeros(moe.moe_balance_workspace_bytes(100, 8, 2, S), dtype=torch.uint8, device=DEV)
        off = torch.tensor(seq, dtype=torch.int32, device=DEV)
        moe.moe_balance_loss(l.to(DEV), idx.to(DEV), 1.0, loss, pad[1:S + 1], slope[1:S + 1], ws, seq_offsets=off)
        d = torch.empty(100, 8, device=DEV)
        moe.moe_gate_backward(l.to(DEV), d, slope=slope[1:S + 1], d_loss=loss, seq_offsets=off)
        torch.cuda.synchronize()
        for t in (pad, slope):
            assert (t[0] == 7).all() and (t[S + 1] == 7).all()


def test_gradient_of_the_loss_by_differences(moe):
    """The whole balance loss, counts fixed, by central differences in float64."""
    T, E, K, h = 40, 6, 2, 1e-4
    l = make_logits(T, E, torch.float32, seed=9)
    idx = torch.argsort(l, dim=1, descending=True)[:, :K].contiguous()
    seq = [0, 13, 40]
    for score in ("softmax", "sigmoid"):
        loss, counts, slope = run_balance(moe, l, idx, seq, 3.0, score)
        d = torch.empty(T, E, device=DEV)
        moe.moe_gate_backward(l.to(DEV), d, slope=slope.to(DEV), d_loss=torch.ones(1, device=DEV),
                              seq_offsets=torch.tensor(seq, dtype=torch.int32, device=DEV),
                              opts=moe.gate_options(score=score))
        for t, e in ((0, 0), (12, 3), (13, 5), (39, 1)):
            x = l.double()
            a, b = x.clone(), x.clone()
            a[t, e] += h
            b[t, e] -= h
            fd = (ref_balance(a, idx, seq, 3.0, score, None)[0] - ref_balance(b, idx, seq, 3.0, score, None)[0]) / (2 * h)
            assert abs(float(d[t, e]) - fd) <= 1e-8 + 4 * (2 * (spread(l) + 4) + E + 48) * U * 2 * float(slope.max())


def test_repeatable_on_streams_and_in_graphs(moe):
    """Two streams at once with a workspace each give the bits of one; a graph of
    the whole router, replayed with other inputs and eager work between, too."""
    T, E, K, S = 513, 128, 8, 3
    ls = [make_logits(T, E, torch.float32, seed=s).to(DEV) for s in range(3)]
    seq = torch.tensor([0, 100, 400, T], dtype=torch.int32, device=DEV)
    n = moe.moe_balance_workspace_bytes(T, E, K, S)
    dw = torch.randn(T, K, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    one = torch.ones(1, device=DEV)

    def buffers():
        return dict(l=torch.empty(T, E, device=DEV), idx=torch.empty(T, K, dtype=torch.int64, device=DEV),
                    w=torch.empty(T, K, device=DEV), loss=torch.empty(1, device=DEV),
                    counts=torch.empty(S, E, dtype=torch.int32, device=DEV), slope=torch.empty(S, E, device=DEV),
                    d=torch.empty(T, E, device=DEV), ws=torch.empty(n, dtype=torch.uint8, device=DEV))

    def step(b, stream=None):
        moe.moe_gate(b["l"], b["idx"], b["w"], stream=stream)
        moe.moe_balance_loss(b["l"], b["idx"], 0.01, b["loss"], b["counts"], b["slope"], b["ws"], seq_offsets=seq,
                             stream=stream)
        moe.moe_gate_backward(b["l"], b["d"], topk_idx=b["idx"], d_topk_w=dw, slope=b["slope"], d_loss=one,
                              seq_offsets=seq, stream=stream)

    outs = ("idx", "w", "loss", "counts", "slope", "d")
    refs = []
    for l in ls:
        b = buffers()
        b["l"].copy_(l)
        step(b)
        refs.append({k: b[k].clone() for k in outs})
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    pair = [buffers() for _ in range(2)]
    for k in range(2):
        pair[k]["l"].copy_(ls[k])
    torch.cuda.synchronize()
    for _ in range(5):
        for k in range(2):
            step(pair[k], streams[k])
    torch.cuda.synchronize()
    for k in range(2):
        for o in outs:
            assert torch.equal(pair[k][o], refs[k][o]), o

    b, e = buffers(), buffers()
    b["l"].copy_(ls[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(b)
    for rep in range(6):
        b["l"].copy_(ls[rep % 3])
        e["l"].copy_(ls[(rep + 1) % 3])
        for o in outs:
            b[o].fill_(3)
        b["ws"].fill_(0x5A)
        step(e)
        g.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert torch.equal(b[o], refs[rep % 3][o]), (rep, o)
            assert torch.equal(e[o], refs[(rep + 1) % 3][o]), (rep, o)
