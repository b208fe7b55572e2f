"""The router and the 8-bit products as a layer uses them, forward and backward,
with the framework's own dispatch and combine between: gate -> balance loss ->
dispatch (bf16 pool) -> quantise -> product -> SwiGLU -> quantise -> product ->
combine, then the gradients of the second product, the routing weights and the
logits.  Every step is checked against float64 on that step's own inputs, so
the bounds are those of the single operators: a product errs by at most 2^-10
of the sum of its |terms| plus half a bf16 step, 2^-8; the combine by K float32
adds and half a bf16 step.
"""
import numpy as np
import pytest
import torch

from tests.test_gpu_block8 import ref_columns, ref_rows, ref_weights, up, values, weight_values
from tests.test_gpu_router import check_balance, check_grad, ref_balance, ref_gate, ref_grad

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
BF = torch.bfloat16


@pytest.fixture(scope="module")
def moe():
    import combine_dispatch_amd as m
    m.lib()
    return m


def close(got, a, b):
    """got against a @ b in float64 with the products' bound."""
    ref, most = a @ b, a.abs() @ b.abs()
    assert ((got.double() - ref).abs() <= 2.0 ** -10 * most + 2.0 ** -8 * ref.abs()).all()


class Layer:
    def __init__(self, moe, T, H, I, E, K, masked, seed=1):
        g = torch.Generator().manual_seed(seed)
        self.m, self.T, self.H, self.I, self.E, self.K = moe, T, H, I, E, K
        self.x = torch.randn(T, H, generator=g).to(BF)
        self.wr = torch.randn(H, E, generator=g) / H ** 0.5
        self.w1 = (torch.randn(E, 2 * I, H, generator=g) / H ** 0.5).to(BF)
        self.w2 = (torch.randn(E, H, I, generator=g) / I ** 0.5).to(BF)
        self.dy = torch.randn(T, H, generator=g).to(BF)
        self.mask = (torch.rand(T, generator=g) >= masked).to(torch.uint8)
        self.logits = self.x.float() @ self.wr
        self.logits[:, E // 2] = -np.inf  # an expert that is out
        self.c1, self.s1 = self.weights(self.w1)[:2]
        self.c2, self.s2, self.c2t, self.s2t = self.weights(self.w2)
        R, Rp = T * K, moe.moe_padded_rows(T * K, E)
        e = lambda *s, dt: torch.empty(s, dtype=dt, device=DEV)
        u8, f32, i32 = torch.uint8, torch.float32, torch.int32
        self.d = dict(
            logits=self.logits.to(DEV), x=self.x.to(DEV), mask=self.mask.to(DEV), dy=self.dy.to(DEV),
            idx=e(T, K, dt=torch.int64), w=e(T, K, dt=f32), loss=e(1, dt=f32), counts=e(1, E, dt=i32), slope=e(1, E, dt=f32),
            bws=e(moe.moe_balance_workspace_bytes(T, E, K), dt=u8), dcounts=e(E, dt=i32), off=e(E + 1, dt=i32),
            src=e(R, dt=i32), slot=e(R, dt=i32), pw=e(R, dt=f32), pool=torch.zeros((R, H), dtype=BF, device=DEV),
            dws=e(moe.moe_dispatch_workspace_bytes(T, H, E, K), dt=u8),
            a=e(R, H, dt=u8), sa=e(H // 128, R, dt=f32), l1=torch.zeros((R, 2 * I), dtype=BF, device=DEV),
            h=e(R, I, dt=BF), b=e(R, up(I), dt=u8), sb=e(up(I) // 128, R, dt=f32), l2=torch.zeros((R, H), dtype=BF, device=DEV),
            y=e(T, H, dt=BF), g=e(R, H, dt=BF), gq=e(R, H, dt=u8), gs=e(H // 128, R, dt=f32),
            dh=torch.zeros((R, I), dtype=BF, device=DEV), gt=e(H, Rp, dt=u8), gts=e(Rp // 128, H, dt=u8),
            ht=e(I, Rp, dt=u8), hts=e(Rp // 128, I, dt=u8), dw2=e(E, H, I, dt=BF), dtw=e(T, K, dt=f32),
            dlogits=e(T, E, dt=f32), one=torch.ones(1, device=DEV))

    def weights(self, w):
        E, N, K = w.shape
        o = [torch.empty(s, dtype=t, device=DEV) for s, t in (
            ((E, N, up(K)), torch.uint8), ((E, up(N) // 128, up(K) // 128), torch.float32),
            ((E, K, up(N)), torch.uint8), ((E, up(K) // 128, up(N) // 128), torch.float32))]
        self.m.moe_quantise_weights(w.to(DEV), *o[:2], codes_t=o[2], scales_t=o[3])
        return o

    def forward(self):
        m, d = self.m, self.d
        m.moe_gate(d["logits"], d["idx"], d["w"], token_mask=d["mask"])
        m.moe_balance_loss(d["logits"], d["idx"], 0.01, d["loss"], d["counts"], d["slope"], d["bws"], token_mask=d["mask"])
        m.moe_dispatch(d["x"], d["idx"], d["w"], self.E, m.MOE_PAYLOAD_BF16, d["dcounts"], d["off"], d["src"], d["slot"],
                       d["pw"], d["pool"], None, d["dws"])
        used = d["off"][self.E:]
        m.moe_quantise_rows(d["pool"], d["a"], d["sa"], rows_used=used)
        m.moe_block_gemm(d["a"], d["sa"], self.c1, self.s1, d["l1"], offsets=d["off"])
        gate, upp = d["l1"][:, :self.I].float(), d["l1"][:, self.I:].float()
        d["h"].copy_(torch.nn.functional.silu(gate) * upp)
        m.moe_quantise_rows(d["h"], d["b"], d["sb"], rows_used=used)
        m.moe_block_gemm(d["b"], d["sb"], self.c2, self.s2, d["l2"], offsets=d["off"])
        m.moe_combine(d["l2"], d["slot"], self.T, self.K, d["y"], topk_w=d["w"])

    def backward(self):
        """Gradients of sum(dy * y) + loss by h, w2, topk_w and the logits."""
        m, d = self.m, self.d
        slot = d["slot"].long().view(self.T, self.K)
        live = slot >= 0
        rows = d["dy"].float()[:, None] * d["w"][:, :, None]
        d["g"].zero_()
        d["g"][slot[live]] = rows[live].to(BF)
        d["dtw"].copy_(torch.where(live, (d["dy"].float()[:, None] * d["l2"].float()[slot.clamp_min(0)]).sum(2), 0.0))
        used = d["off"][self.E:]
        m.moe_quantise_rows(d["g"], d["gq"], d["gs"], rows_used=used)
        m.moe_block_gemm(d["gq"], d["gs"], self.c2t, self.s2t, d["dh"], offsets=d["off"])
        m.moe_quantise_columns(d["g"], d["gt"], d["gts"], offsets=d["off"])
        m.moe_quantise_columns(d["h"], d["ht"], d["hts"], offsets=d["off"])
        m.moe_block_gemm_wgrad(d["gt"], d["gts"], d["ht"], d["hts"], d["dw2"], rows=self.T * self.K, offsets=d["off"])
        m.moe_gate_backward(d["logits"], d["dlogits"], topk_idx=d["idx"], d_topk_w=d["dtw"], slope=d["slope"],
                            d_loss=d["one"], token_mask=d["mask"])


@pytest.mark.parametrize("T,H,I,E,K,masked", [(200, 256, 136, 8, 2, 0.2), (37, 512, 264, 16, 4, 0.0), (600, 256, 128, 4, 2, 0.5),
                                              (1, 256, 128, 6, 3, 0.0), (5, 256, 128, 4, 2, 1.0)])
def test_layer_forward_and_backward(moe, T, H, I, E, K, masked):
    L = Layer(moe, T, H, I, E, K, masked)
    L.forward()
    L.backward()
    d = {k: v.cpu() for k, v in L.d.items()}
    idx, w = ref_gate(L.logits, K, "softmax", True, 1.0, None, L.mask)
    assert torch.equal(d["idx"], idx)
    check_balance((d["loss"], d["counts"], d["slope"]), ref_balance(L.logits, idx, [0, T], 0.01, "softmax", L.mask), L.logits, E)
    # the dispatch counts what the loss counted, and leaves out the padding
    assert torch.equal(d["dcounts"], d["counts"][0])
    off = d["off"].tolist()
    assert off[E] == int((idx >= 0).sum())
    flat = idx.view(-1)
    order = torch.tensor([s for e in range(E) for s in torch.nonzero(flat == e).view(-1).tolist()], dtype=torch.long)
    assert torch.equal(d["pool"][:off[E]], L.x[order // K])
    w1v, w2v, w2tv = weight_values(L.c1, L.s1), weight_values(L.c2, L.s2), weight_values(L.c2t, L.s2t)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            assert (d["dw2"][e] == 0).all()
            continue
        ca, sa = ref_rows(d["pool"][lo:hi])
        assert torch.equal(d["a"][lo:hi], ca)
        close(d["l1"][lo:hi], values(ca, sa), w1v[e].t().contiguous())
        cb, sb = ref_rows(d["h"][lo:hi])
        assert torch.equal(d["b"][lo:hi], cb)
        close(d["l2"][lo:hi], values(cb, sb), w2v[e].t().contiguous())
        cg, sg = ref_rows(d["g"][lo:hi])
        close(d["dh"][lo:hi], values(cg, sg), w2tv[e].t().contiguous()[:, :I])

        def columns(v):
            c, s = ref_columns(v, [hi - lo])
            return c.view(torch.float8_e4m3fn).double() * torch.exp2(s.double() - 127).t().repeat_interleave(128, 1)

        close(d["dw2"][e], columns(d["g"][lo:hi]), columns(d["h"][lo:hi]).t().contiguous())
    assert (d["l1"][off[E]:] == 0).all() and (d["l2"][off[E]:] == 0).all() and (d["dh"][off[E]:] == 0).all()
    terms = torch.zeros(T, K, H, dtype=torch.float64)
    terms.view(T * K, H)[order] = d["l2"][:off[E]].double()
    terms *= d["w"].double()[:, :, None]
    y = terms.sum(1)
    assert ((d["y"].double() - y).abs() <= 2.0 ** -8 * y.abs() + (K + 1) * 2.0 ** -24 * terms.abs().sum(1)).all()
    ref, mag = ref_grad(L.logits, idx, d["dtw"], "softmax", True, 1.0, d["slope"], np.float32(1), [0, T], L.mask)
    check_grad(d["dlogits"], ref, mag, L.logits, E)


def test_layer_in_a_graph(moe):
    """The whole chain captured once, replayed over other tokens and routings."""
    args = (150, 256, 128, 8, 2, 0.1)
    layers = [Layer(moe, *args, seed=s) for s in (1, 2, 3)]
    refs = []
    keep = ("y", "loss")
    for L in layers:
        L.c1, L.s1, L.c2, L.s2, L.c2t, L.s2t = (getattr(layers[0], k) for k in ("c1", "s1", "c2", "s2", "c2t", "s2t"))
        L.forward()
        refs.append({k: L.d[k].clone() for k in keep})
    L = Layer(moe, *args, seed=1)
    L.c1, L.s1, L.c2, L.s2, L.c2t, L.s2t = (getattr(layers[0], k) for k in ("c1", "s1", "c2", "s2", "c2t", "s2t"))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.forward()
    for rep in range(6):
        src = layers[rep % 3]
        for k in ("logits", "x", "mask"):
            L.d[k].copy_(src.d[k])
        for k in ("y", "loss", "l1", "l2", "pool"):
            L.d[k].fill_(3)
        layers[(rep + 1) % 3].forward()  # eager work between
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(L.d["y"], refs[rep % 3]["y"]) and torch.equal(L.d["loss"], refs[rep % 3]["loss"]), rep
        assert torch.equal(layers[(rep + 1) % 3].d["y"], refs[(rep + 1) % 3]["y"])
