"""GPU tests of the 8-bit block products (include/moe_block8.h).

Quantisers: the same float32 arithmetic in torch on the CPU, bit for bit.

Products, two ways:
 - Exact: codes in {-1, 0, 1}, scales powers of two.  Every partial sum is a
   small multiple of a power of two, so the float32 sums are exact whatever
   their order and the one rounding to bf16 decides every bit.
 - Random codes and scales against float64 sums of the same values:
   |error| <= 2^-10 sum |a w| + 2^-8 |result|.  The first term is the matrix
   core's: inside 8 consecutive k it drops what lies below 2^-13 of the
   largest product, less than 7 * 2^-13 < 2^-10.19 of the run's products, and
   the float32 adds of at most 64 blocks (64 * 2^-24) fit in what is left; the
   second is half a step of bf16.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn
MIN = 2.0 ** -126


@pytest.fixture(scope="module")
def moe():
    import combine_dispatch_amd as m
    m.lib()
    return m


def up(n, m=128):
    return (n + m - 1) // m * m


def pad(x, rows, cols):
    out = torch.zeros((*x.shape[:-2], rows, cols), dtype=x.dtype)
    out[..., :x.shape[-2], :x.shape[-1]] = x
    return out


def amax448(v, dims):
    s = v.abs().amax(dims) / 448.0
    return torch.where(s < MIN, torch.full_like(s, MIN), s)


def ref_rows(x):
    R, C = x.shape
    v = pad(x.float(), R, up(C)).view(R, -1, 128)
    s = amax448(v, 2)
    return (v * (1 / s)[:, :, None]).to(E4M3).view(torch.uint8).view(R, -1), s.t().contiguous()


def ref_weights(w):
    E, N, K = w.shape
    v = pad(w.float(), up(N), up(K)).view(E, up(N) // 128, 128, up(K) // 128, 128)
    s = amax448(v, (2, 4))
    q = (v * (1 / s)[:, :, None, :, None]).to(E4M3).view(torch.uint8).reshape(E, up(N), up(K))
    return q, s


def ref_columns(x, sizes):
    """codes [C][R'], UE8M0 bytes [R'/128][C] of the groups' blocks, in order."""
    C = x.shape[1]
    codes, scales, at = [], [], 0
    for n in sizes:
        if n:
            v = pad(x[at:at + n].float(), up(n), C).view(-1, 128, C)
            a = v.abs().amax(1)
            b = torch.clamp((a.view(torch.int32) >> 23) - 8 + ((a.view(torch.int32) & 0x7FFFFF) > 0x600000), 1, 254)
            inv = ((254 - b) << 23).to(torch.int32).view(torch.float32)
            codes.append((v * inv[:, None, :]).to(E4M3).view(torch.uint8).view(-1, C))
            scales.append(b.to(torch.uint8))
        at += n
    return torch.cat(codes).t().contiguous(), torch.cat(scales)


def data(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g) * torch.exp(torch.randn(shape[-1], generator=g)) * scale
    return x.to(dtype)


def offsets_of(sizes):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device=DEV)


# ---- quantisers --------------------------------------------------------------------

@pytest.mark.parametrize("R,C", [(1, 1), (1, 128), (3, 7), (32, 512), (33, 520), (31, 640), (100, 129), (65, 2000), (7, 1001)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantise_rows(moe, R, C, dtype):
    x = data((R, C), dtype, R + C)
    x[0] = 0  # a block of zeros
    codes = torch.full((R, up(C)), 77, dtype=torch.uint8, device=DEV)
    scales = torch.full((up(C) // 128, R), 7.0, device=DEV)
    moe.moe_quantise_rows(x.to(DEV), codes, scales)
    rc, rs = ref_rows(x)
    assert torch.equal(scales.cpu(), rs)
    assert torch.equal(codes.cpu(), rc)


def test_quantise_rows_used_and_unaligned(moe):
    """Rows at or past *rows_used stay as they were; a view off the 16-byte
    boundary takes the narrow loads."""
    R, C = 70, 256
    for used in (0, 1, 33, 64, 69, 70, 1000, -3):
        x = data((1, 1 + R * C), torch.bfloat16, used + 9).view(-1)[1:].view(R, C)
        dx = x.to(DEV)
        base = torch.empty(1 + R * C, dtype=torch.bfloat16, device=DEV)
        base[1:].copy_(dx.view(-1))
        codes = torch.full((R, C), 77, dtype=torch.uint8, device=DEV)
        scales = torch.full((2, R), 7.0, device=DEV)
        moe.moe_quantise_rows(base[1:].view(R, C), codes, scales,
                              rows_used=torch.tensor([used], dtype=torch.int32, device=DEV))
        n = min(max(used, 0), R)
        rc, rs = ref_rows(x)
        assert torch.equal(codes[:n].cpu(), rc[:n]) and (codes[n:] == 77).all()
        assert torch.equal(scales[:, :n].cpu(), rs[:, :n]) and (scales[:, n:] == 7).all()


@pytest.mark.parametrize("value", [float("inf"), float("nan"), -float("inf")])
def test_quantise_rows_bad_values_show_in_the_scale(moe, value):
    x = data((4, 384), torch.float32, 1)
    x[2, 130] = value
    codes = torch.empty((4, 384), dtype=torch.uint8, device=DEV)
    scales = torch.empty((3, 4), device=DEV)
    moe.moe_quantise_rows(x.to(DEV), codes, scales)
    bad = torch.zeros(3, 4, dtype=torch.bool)
    bad[1, 2] = True
    assert torch.equal(~torch.isfinite(scales.cpu()), bad)
    rc, rs = ref_rows(torch.where(torch.isfinite(x), x, torch.zeros(())))
    assert torch.equal(codes.cpu()[:2], rc[:2]) and torch.equal(codes.cpu()[2, :128], rc[2, :128])
    # and the column form: the UE8M0 NaN
    cc = torch.empty((384, 128), dtype=torch.uint8, device=DEV)
    cs = torch.empty((1, 384), dtype=torch.uint8, device=DEV)
    moe.moe_quantise_columns(x.to(DEV), cc, cs)
    assert int(cs[0, 130]) == 255 and int((cs == 255).sum()) == 1


def test_quantise_extreme_magnitudes(moe):
    """Subnormal blocks are held at the smallest scale, the largest finite ones below an infinite scale."""
    x = torch.zeros(6, 128)
    x[0, 3], x[1, 3], x[2, 3], x[3, 3] = 1e-45, 2.0 ** -126, 3e38, -3.4028234663852886e38
    x[4, 3], x[5, :] = 448 * 2.0 ** -126, 1.7
    codes = torch.empty((6, 128), dtype=torch.uint8, device=DEV)
    scales = torch.empty((1, 6), device=DEV)
    moe.moe_quantise_rows(x.to(DEV), codes, scales)
    rc, rs = ref_rows(x)
    assert torch.equal(codes.cpu(), rc) and torch.equal(scales.cpu(), rs)
    for r in range(6):
        cc = torch.empty((128, 128), dtype=torch.uint8, device=DEV)
        cs = torch.empty((1, 128), dtype=torch.uint8, device=DEV)
        moe.moe_quantise_columns(x[r:r + 1].to(DEV), cc, cs)
        rc, rs = ref_columns(x[r:r + 1], [1])
        assert torch.equal(cc.cpu(), rc) and torch.equal(cs.cpu(), rs)


@pytest.mark.parametrize("E,N,K", [(1, 1, 1), (2, 128, 128), (3, 130, 260), (1, 1001, 72), (2, 7, 640), (1, 256, 1000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("both", [True, False])
def test_quantise_weights(moe, E, N, K, dtype, both):
    w = data((E, N, K), dtype, N + K, 0.02)
    w[0, :128, :128] = 0
    codes = torch.full((E, N, up(K)), 77, dtype=torch.uint8, device=DEV)
    scales = torch.full((E, up(N) // 128, up(K) // 128), 7.0, device=DEV)
    ct = torch.full((E, K, up(N)), 77, dtype=torch.uint8, device=DEV) if both else None
    st = torch.full((E, up(K) // 128, up(N) // 128), 7.0, device=DEV) if both else None
    moe.moe_quantise_weights(w.to(DEV), codes, scales, codes_t=ct, scales_t=st)
    rc, rs = ref_weights(w)
    assert torch.equal(scales.cpu(), rs)
    assert torch.equal(codes.cpu(), rc[:, :N])
    if both:
        assert torch.equal(ct.cpu(), rc.transpose(1, 2)[:, :K])
        assert torch.equal(st.cpu(), rs.transpose(1, 2))


@pytest.mark.parametrize("sizes", [[1], [128], [300], [0, 5, 0, 128, 129, 0], [1] * 40, [0, 0, 260]])
@pytest.mark.parametrize("C", [1, 8, 128, 130, 1000])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_quantise_columns(moe, sizes, C, dtype):
    R, E = sum(sizes), len(sizes)
    x = data((R, C), dtype, R + C)
    Rp = moe.moe_padded_rows(R, E)
    codes = torch.full((C, Rp), 77, dtype=torch.uint8, device=DEV)
    scales = torch.full((Rp // 128, C), 7, dtype=torch.uint8, device=DEV)
    moe.moe_quantise_columns(x.to(DEV), codes, scales, offsets=None if E == 1 else offsets_of(sizes))
    rc, rs = ref_columns(x, sizes)
    used = rc.shape[1]
    assert torch.equal(scales[:used // 128].cpu(), rs) and torch.equal(codes[:, :used].cpu(), rc)
    assert (codes[:, used:] == 77).all() and (scales[used // 128:] == 7).all()


# ---- products ------------------------------------------------------------------------

def exact_codes(shape, seed, density):
    """e4m3 codes of -1, 0 and 1."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randint(0, 2, shape, generator=g) * 2 - 1
    keep = torch.rand(shape, generator=g) < density
    return (v * keep).float()


def code(v):
    return v.to(E4M3).view(torch.uint8).to(DEV)


def run_product(moe, a, sa, w, sw, sizes, R, N, fill=-3.0, dense=False):
    """out with a guard row on each side of the R rows."""
    buf = torch.full((R + 2, N), fill, dtype=torch.bfloat16, device=DEV)
    out = buf[1:R + 1]
    moe.moe_block_gemm(a, sa, w, sw, out, offsets=None if dense else offsets_of(sizes))
    assert (buf[0] == fill).all() and (buf[R + 1] == fill).all()
    return out


def values(a, sa):
    R, K = a.shape
    return a.cpu().view(E4M3).double() * sa.cpu().double().t().repeat_interleave(128, 1)[:, :K]


def weight_values(w, sw):
    E, N, K = w.shape
    return w.cpu().view(E4M3).double() * sw.cpu().double().repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)


SHAPES = [  # group sizes, N, K (and the kernels they meet: few and many rows a group)
    ([1], 8, 128), ([1], 1001, 256), ([5], 128, 384), ([64], 96, 128), ([65], 257, 640), ([130], 40, 256),
    ([255, 0, 257], 264, 384), ([0, 0, 3], 520, 128), ([7, 0, 63, 1, 64, 65], 130, 896), ([1] * 33, 72, 256),
    ([300, 20, 0, 511], 300, 512), ([1000], 1000, 1024), ([2, 700], 17, 128)]


@pytest.mark.parametrize("sizes,N,K", SHAPES)
def test_product_exact(moe, sizes, N, K):
    R, E = sum(sizes), len(sizes)
    a = exact_codes((R, K), 1, 0.5)
    w = exact_codes((E, N, K), 2, 0.25)
    g = torch.Generator().manual_seed(3)
    sa = torch.exp2(torch.randint(-2, 3, (K // 128, R), generator=g).float())
    sw = torch.exp2(torch.randint(-2, 3, (E, up(N) // 128, K // 128), generator=g).float())
    ca, cw = code(a), code(w)
    out = run_product(moe, ca, sa.to(DEV), cw, sw.to(DEV), sizes, R, N)
    va, vw = values(ca, sa), weight_values(cw, sw)
    at = 0
    for e, n in enumerate(sizes):
        ref = va[at:at + n] @ vw[e].t().contiguous()
        assert torch.equal(out[at:at + n].cpu(), ref.float().to(torch.bfloat16)), e
        at += n


@pytest.mark.parametrize("sizes,N,K", SHAPES)
def test_product_random(moe, sizes, N, K):
    R, E = sum(sizes), len(sizes)
    ca, sa = ref_rows(data((R, K), torch.float32, 5))
    cw, sw = ref_weights(data((E, N, K), torch.float32, 6, 0.02))
    cw = cw[:, :N].contiguous()
    out = run_product(moe, ca.to(DEV), sa.to(DEV), cw.to(DEV), sw.to(DEV), sizes, R, N).cpu().double()
    va, vw = values(ca, sa), weight_values(cw, sw)
    at = 0
    for e, n in enumerate(sizes):
        ref = va[at:at + n] @ vw[e].t().contiguous()
        most = va[at:at + n].abs() @ vw[e].abs().t().contiguous()
        assert ((out[at:at + n] - ref).abs() <= 2.0 ** -10 * most + 2.0 ** -8 * ref.abs()).all()
        at += n


def test_product_dense_and_rows_outside(moe):
    """Without offsets all rows are one group; rows before the first and behind
    the last offset stay as they were."""
    R, N, K = 200, 136, 256
    ca, sa = ref_rows(data((R, K), torch.bfloat16, 5))
    cw, sw = ref_weights(data((2, N, K), torch.bfloat16, 6, 0.02))
    cw = cw[:, :N].contiguous().to(DEV)
    ca, sa, sw = ca.to(DEV), sa.to(DEV), sw.to(DEV)
    dense = run_product(moe, ca, sa, cw[:1].contiguous(), sw[:1].contiguous(), None, R, N, dense=True)
    one = run_product(moe, ca, sa, cw[:1].contiguous(), sw[:1].contiguous(), [R], R, N)
    assert torch.equal(dense, one)
    for off in ([20, 50, 170], [0, 0, 0], [200, 200, 200], [10, 10, 11]):
        out = torch.full((R, N), -3.0, dtype=torch.bfloat16, device=DEV)
        moe.moe_block_gemm(ca, sa, cw, sw, out, offsets=torch.tensor(off, dtype=torch.int32, device=DEV))
        assert (out[:off[0]] == -3).all() and (out[off[2]:] == -3).all()
        # the same bits as in the dense product, row by row
        assert torch.equal(out[off[0]:off[1]], dense[off[0]:off[1]])
        assert (out[off[1]:off[2]] != -3).any(1).all()


@pytest.mark.parametrize("R", [40, 150, 3000])  # split K, small tiles, large tiles
def test_products_bad_offsets_do_nothing(moe, R):
    """Out of order or out of range: no call reads past its arrays, none writes."""
    N, K, E = 64, 128, 3
    ca, sa = ref_rows(data((R, K), torch.bfloat16, 5))
    cw, sw = ref_weights(data((E, N, K), torch.bfloat16, 6))
    cw = cw[:, :N].contiguous().to(DEV)
    Rp = moe.moe_padded_rows(R, E)
    x = data((R, N), torch.bfloat16, 1).to(DEV)
    for off in ([0, R, 20, R], [-9, R, R, R], [0, 5, 9, R + 1], [1 << 30, 1 << 30, 1 << 30, 1 << 30], [0, R, 0, R],
                [-(1 << 31), 0, 0, R], [0, 0, 0, (1 << 31) - 1]):
        o = torch.tensor(off, dtype=torch.int32, device=DEV)
        out = torch.full((R, N), -3.0, dtype=torch.bfloat16, device=DEV)
        moe.moe_block_gemm(ca.to(DEV), sa.to(DEV), cw, sw.to(DEV), out, offsets=o)
        codes = torch.full((N, Rp), 77, dtype=torch.uint8, device=DEV)
        scales = torch.full((Rp // 128, N), 99, dtype=torch.uint8, device=DEV)
        moe.moe_quantise_columns(x, codes, scales, offsets=o)
        dw = torch.full((E, N, N), -3.0, dtype=torch.bfloat16, device=DEV)
        moe.moe_block_gemm_wgrad(codes, scales, codes, scales, dw, rows=R, offsets=o)
        for t, v in ((out, -3), (codes, 77), (scales, 99), (dw, -3)):
            assert (t == v).all(), off


def test_product_of_bad_blocks_is_nan(moe):
    """An infinity in one block of the input reaches that row's outputs only."""
    R, N, K = 70, 40, 256
    x = data((R, K), torch.float32, 5)
    x[33, 200] = float("inf")
    codes = torch.empty((R, K), dtype=torch.uint8, device=DEV)
    scales = torch.empty((2, R), device=DEV)
    moe.moe_quantise_rows(x.to(DEV), codes, scales)
    cw, sw = ref_weights(data((1, N, K), torch.float32, 6))
    out = torch.empty((R, N), dtype=torch.bfloat16, device=DEV)
    moe.moe_block_gemm(codes, scales, cw[:, :N].contiguous().to(DEV), sw.to(DEV), out)
    assert not torch.isfinite(out[33]).any()
    assert torch.isfinite(out[:33]).all() and torch.isfinite(out[34:]).all()


WGRAD = [([1], 8, 8), ([128], 128, 128), ([130], 257, 300), ([0, 300, 0, 5], 130, 72), ([129, 127, 1], 40, 1001),
         ([1] * 20, 64, 136), ([700, 0, 400], 256, 264), ([0, 0], 24, 40)]


# enough 256 x 256 tiles for the large kernel (the sets above have too few of them), one and two rounds of them
MIXED = [1, 128, 130, 0, 300, 5, 129, 127, 257, 0, 1, 1, 2, 3, 64, 400, 33]
# and small tiles of which a workgroup has several, most without rows
WGRAD_EMPTY = [([0] * 5 + [7] + [0] * 40 + [13] + [0] * 17, 300, 300), ([0] * 150 + [260] + [0] * 149 + [30] + [0] * 6, 100, 72)]
WGRAD_LARGE = [(MIXED, 700, 760), (MIXED, 760, 761), ([128] + [0, 1, 140] * 13, 701, 768)]


@pytest.mark.parametrize("sizes,N,K", WGRAD + WGRAD_LARGE + WGRAD_EMPTY)
def test_wgrad_exact(moe, sizes, N, K):
    """Values of -1, 0, 1 times a power of two per column: exact sums."""
    R, E = sum(sizes), len(sizes)
    g = torch.Generator().manual_seed(3)
    dy = exact_codes((R, N), 1, 0.5) * torch.exp2(torch.randint(-3, 4, (1, N), generator=g).float())
    x = exact_codes((R, K), 2, 0.3) * torch.exp2(torch.randint(-3, 4, (1, K), generator=g).float())
    off = offsets_of(sizes)
    Rp = moe.moe_padded_rows(R, E)

    def columns(v):
        c = torch.empty((v.shape[1], Rp), dtype=torch.uint8, device=DEV)
        s = torch.empty((Rp // 128, v.shape[1]), dtype=torch.uint8, device=DEV)
        moe.moe_quantise_columns(v.to(DEV), c, s, offsets=off)
        return c, s

    buf = torch.full((E * N + 2, K), -3.0, dtype=torch.bfloat16, device=DEV)
    out = buf[1:E * N + 1].view(E, N, K)
    moe.moe_block_gemm_wgrad(*columns(dy), *columns(x), out, rows=R, offsets=off)
    assert (buf[0] == -3).all() and (buf[E * N + 1] == -3).all()
    at = 0
    for e, n in enumerate(sizes):
        ref = dy[at:at + n].double().t().contiguous() @ x[at:at + n].double()
        assert torch.equal(out[e].cpu(), ref.float().to(torch.bfloat16)), e
        at += n


@pytest.mark.parametrize("sizes,N,K", WGRAD[:-1] + WGRAD_LARGE[:2])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_wgrad_random(moe, sizes, N, K, dtype):
    R, E = sum(sizes), len(sizes)
    dy, x = data((R, N), dtype, 1, 1e-3), data((R, K), dtype, 2)
    (cg, sg), (cx, sx) = ref_columns(dy, sizes), ref_columns(x, sizes)
    Rp, used = moe.moe_padded_rows(R, E), cg.shape[1]

    def full(c, s):
        fc = torch.full((c.shape[0], Rp), 0x7F, dtype=torch.uint8)  # NaN behind the last group: never read
        fs = torch.full((Rp // 128, c.shape[0]), 255, dtype=torch.uint8)
        fc[:, :used], fs[:used // 128] = c, s
        return fc.to(DEV), fs.to(DEV)

    out = torch.empty((E, N, K), dtype=torch.bfloat16, device=DEV)
    moe.moe_block_gemm_wgrad(*full(cg, sg), *full(cx, sx), out, rows=R, offsets=offsets_of(sizes))

    def decode(c, s):
        return c.view(E4M3).double() * torch.exp2(s.double() - 127).t().repeat_interleave(128, 1)

    vg, vx = decode(cg, sg), decode(cx, sx)
    at = 0
    for e, n in enumerate(sizes):
        a, b = vg[:, at:at + up(n)], vx[:, at:at + up(n)].t().contiguous()
        ref, most = a @ b, a.abs() @ b.abs()
        got = out[e].cpu().double()
        assert ((got - ref).abs() <= 2.0 ** -10 * most + 2.0 ** -8 * ref.abs()).all()
        at += up(n)


def test_wgrad_without_rows_writes_zeros(moe):
    e = torch.empty((16, 0), dtype=torch.uint8, device=DEV)
    s = torch.empty((0, 16), dtype=torch.uint8, device=DEV)
    out = torch.full((1, 16, 16), -3.0, dtype=torch.bfloat16, device=DEV)
    moe.moe_block_gemm_wgrad(e, s, e, s, out, rows=0)
    assert (out == 0).all()


def test_gradients_against_differences(moe):
    """The three products around one another: with L = sum(dy * y), the input's
    and the weights' gradients equal the change of L along a step of either
    (the product is linear, so the difference is exact up to the stated error
    of each product; values whose codes are exact)."""
    sizes, N, K = [70, 0, 200], 128, 256
    R, E = sum(sizes), len(sizes)
    off = offsets_of(sizes)
    x, w = exact_codes((R, K), 1, 0.5), exact_codes((E, N, K), 2, 0.25)
    dy = exact_codes((R, N), 3, 0.2)
    dx_dir, dw_dir = exact_codes((R, K), 4, 0.02), exact_codes((E, N, K), 5, 0.02)

    def rows(v):
        c = torch.empty((R, v.shape[1]), dtype=torch.uint8, device=DEV)
        s = torch.empty((v.shape[1] // 128, R), device=DEV)
        moe.moe_quantise_rows(v.to(DEV), c, s)
        return c, s

    def weights(v):
        c, s = torch.empty((E, N, K), dtype=torch.uint8, device=DEV), torch.empty((E, N // 128, K // 128), device=DEV)
        ct, st = torch.empty((E, K, N), dtype=torch.uint8, device=DEV), torch.empty((E, K // 128, N // 128), device=DEV)
        moe.moe_quantise_weights(v.to(DEV), c, s, codes_t=ct, scales_t=st)
        return c, s, ct, st

    def forward(xv, wv):
        y = torch.empty((R, N), dtype=torch.bfloat16, device=DEV)
        moe.moe_block_gemm(*rows(xv), *weights(wv)[:2], y, offsets=off)
        return (y.double() * dy.to(DEV).double()).sum()

    c, s, ct, st = weights(w)
    gx = torch.empty((R, K), dtype=torch.bfloat16, device=DEV)
    moe.moe_block_gemm(*rows(dy), ct, st, gx, offsets=off)
    Rp = moe.moe_padded_rows(R, E)

    def columns(v):
        q = torch.empty((v.shape[1], Rp), dtype=torch.uint8, device=DEV)
        z = torch.empty((Rp // 128, v.shape[1]), dtype=torch.uint8, device=DEV)
        moe.moe_quantise_columns(v.to(DEV), q, z, offsets=off)
        return q, z

    gw = torch.empty((E, N, K), dtype=torch.bfloat16, device=DEV)
    moe.moe_block_gemm_wgrad(*columns(dy), *columns(x), gw, rows=R, offsets=off)
    # codes of +-448 at a scale of 1/448: values are 1 up to 2^-23, sums below
    # 256, so each bf16 entry is a whole number up to float32 error and rounds to it
    step = forward(x + dx_dir, w) - forward(x, w)
    near = (dx_dir + x).abs().amax() <= 2
    assert near
    want = (gx.double().cpu() * dx_dir.double()).sum()
    # x + dir holds 2s: codes 448 and 224 stand for 2 and 1 exactly as well
    assert abs(float(step) - float(want)) <= 1e-3 * float(dy.abs().sum())
    step = forward(x, w + dw_dir) - forward(x, w)
    want = (gw.double().cpu() * dw_dir.double()).sum()
    assert abs(float(step) - float(want)) <= 1e-3 * float(dy.abs().sum())


def test_other_stream_and_graph(moe):
    """On a stream of the caller's, and captured once and replayed over changed
    inputs and offsets with eager work between: the bits of an eager call."""
    N, K, E, R = 264, 384, 4, 600
    cw, sw = ref_weights(data((E, N, K), torch.bfloat16, 6, 0.02))
    cw, sw = cw[:, :N].contiguous().to(DEV), sw.to(DEV)
    xs = [data((R, K), torch.bfloat16, s).to(DEV) for s in (1, 2, 3)]
    offs = [offsets_of(s) for s in ([100, 0, 500, 0], [0, 0, 0, 600], [1, 298, 300, 1])]

    def buffers():
        Rp = moe.moe_padded_rows(R, E)
        return dict(x=torch.empty((R, K), dtype=torch.bfloat16, device=DEV), off=torch.empty(E + 1, dtype=torch.int32, device=DEV),
                    a=torch.empty((R, K), dtype=torch.uint8, device=DEV), s=torch.empty((K // 128, R), device=DEV),
                    y=torch.empty((R, N), dtype=torch.bfloat16, device=DEV),
                    xc=torch.empty((K, Rp), dtype=torch.uint8, device=DEV), xs=torch.empty((Rp // 128, K), dtype=torch.uint8, device=DEV),
                    yc=torch.empty((N, Rp), dtype=torch.uint8, device=DEV), ys=torch.empty((Rp // 128, N), dtype=torch.uint8, device=DEV),
                    dw=torch.empty((E, N, K), dtype=torch.bfloat16, device=DEV))

    def step(b, stream=None):
        moe.moe_quantise_rows(b["x"], b["a"], b["s"], stream=stream)
        moe.moe_block_gemm(b["a"], b["s"], cw, sw, b["y"], offsets=b["off"], stream=stream)
        moe.moe_quantise_columns(b["x"], b["xc"], b["xs"], offsets=b["off"], stream=stream)
        moe.moe_quantise_columns(b["y"], b["yc"], b["ys"], offsets=b["off"], stream=stream)
        moe.moe_block_gemm_wgrad(b["yc"], b["ys"], b["xc"], b["xs"], b["dw"], rows=R, offsets=b["off"], stream=stream)

    def load(b, i):
        b["x"].copy_(xs[i])
        b["off"].copy_(offs[i])

    refs = []
    for i in range(3):
        b = buffers()
        load(b, i)
        step(b)
        refs.append((b["y"].clone(), b["dw"].clone()))
    torch.cuda.synchronize()
    streams, pair = [torch.cuda.Stream() for _ in range(2)], [buffers() for _ in range(2)]
    for i in range(2):
        load(pair[i], i)
    torch.cuda.synchronize()
    for _ in range(3):
        for i in range(2):
            step(pair[i], streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(pair[i]["y"], refs[i][0]) and torch.equal(pair[i]["dw"], refs[i][1])
    b, e = buffers(), buffers()
    load(b, 0)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step(b)
    for rep in range(6):
        load(b, rep % 3)
        load(e, (rep + 1) % 3)
        b["y"].fill_(5)
        b["dw"].fill_(5)
        step(e)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(b["y"], refs[rep % 3][0]) and torch.equal(b["dw"], refs[rep % 3][1]), rep
        assert torch.equal(e["y"], refs[(rep + 1) % 3][0]) and torch.equal(e["dw"], refs[(rep + 1) % 3][1]), rep


def test_binding_checks(moe):
    a = torch.zeros((4, 128), dtype=torch.uint8, device=DEV)
    s = torch.zeros((1, 4), device=DEV)
    w = torch.zeros((2, 8, 128), dtype=torch.uint8, device=DEV)
    sw = torch.zeros((2, 1, 1), device=DEV)
    out = torch.zeros((4, 8), dtype=torch.bfloat16, device=DEV)
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device=DEV)
    moe.moe_block_gemm(a, s, w, sw, out, offsets=off)
    for args, kw in (((a, s, w, sw, out), {}), ((a, s, w, sw, out.float()), dict(offsets=off)),
                     ((a, s, w[:, :, ::2], sw, out), dict(offsets=off)), ((a, s.t(), w, sw, out), dict(offsets=off)),
                     ((a, s, w, sw, out), dict(offsets=off.long())), ((a, s, w, sw, out.t()), dict(offsets=off)),
                     ((a[:3], s, w, sw, out), dict(offsets=off)), ((a, s, w, sw, out), dict(offsets=off.cpu()))):
        with pytest.raises(moe.MoeError) as err:
            moe.moe_block_gemm(*args, **kw)
        assert err.value.status == moe.MOE_ERR_INVALID_ARG
