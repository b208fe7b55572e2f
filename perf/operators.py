"""Workloads of the expert layer's router and 8-bit products: the top-k gate, the balance loss,
the quantisers to e4m3 with a scale per block of 128, and the grouped product with its gradients.

``own`` chooses between the operators' plain forms in elementary torch operations and the calls
of ``combine_dispatch_amd``; everything else is the same for both.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn
F32_MIN_NORMAL = 2.0 ** -126


# ---- cases ---------------------------------------------------------------------------------------

def listed():
    return [
        # one serving step's router: a handful of tokens, sigmoid scores with a selection bias
        dict(name="gate_decode", kind="gate", T=64, E=256, K=8, dtype="f32", score="sigmoid", renorm=True, bias=True,
             masked=0.0, backward=False),
        # a training batch's router, forward and backward, softmax over 128 experts
        dict(name="gate_train", kind="gate", T=16384, E=128, K=8, dtype="f32", score="softmax", renorm=True, bias=False,
             masked=0.0, backward=True),
        # a padded batch of an odd length in bf16, weights not renormalised (the gradient reaches every expert)
        dict(name="gate_padded_bf16", kind="gate", T=4099, E=32, K=2, dtype="bf16", score="softmax", renorm=False,
             bias=False, masked=0.2, backward=True),
        # the balance loss of a small fine-tuning batch
        dict(name="balance_small", kind="balance", T=509, E=32, K=8, S=1, dtype="bf16", score="softmax", masked=0.1),
        # the same over a training batch of packed sequences, one loss per sequence
        dict(name="balance_sequences", kind="balance", T=16384, E=128, K=8, S=24, dtype="f32", score="sigmoid", masked=0.0),
        # one token through a dense 8-bit projection: the weights stream through once
        dict(name="linear_one_token", kind="linear", R=1, N=4096, K=7168, E=1, skew=0.0, dtype="bf16"),
        # a decoding batch over the experts (128 tokens, 8 experts each): 940 MB of weights for 1024 rows
        dict(name="product_decode", kind="product", R=1024, N=4096, K=7168, E=32, skew=0.0),
        # a prompt over the experts: the L1 product of the prefill workload
        dict(name="product_prefill", kind="product", R=65536, N=4096, K=7168, E=32, skew=0.0),
        # many experts of unequal load, the activations quantised on the way in
        dict(name="linear_many_skewed", kind="linear", R=131072, N=1536, K=2048, E=128, skew=1.2, dtype="bf16"),
        # odd sizes everywhere: a ragged dense product with a partial block of 128 along K and odd N, from float32
        dict(name="linear_odd_f32", kind="linear", R=1733, N=1001, K=2000, E=1, skew=0.0, dtype="f32"),
        # one training step's gradients of a grouped product: the incoming gradient and the inputs are quantised on the way
        dict(name="gradients_many", kind="gradients", R=32768, N=1536, K=2048, E=32, skew=0.6, dtype="bf16"),
        # the weights after an optimiser step: codes for the product and transposed codes for its gradient
        dict(name="weights_requantised", kind="weights", E=32, N=1536, K=2048, dtype="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["gate", "balance", "linear", "product", "gradients", "weights"])
    if kind in ("gate", "balance"):
        T, E = _log_int(rng, 1, 16384), _log_int(rng, 4, 512)
        K = rng.randint(1, min(E, 12))
        c = dict(kind=kind, T=T, E=E, K=K, dtype=rng.choice(["f32", "bf16"]), score=rng.choice(["softmax", "sigmoid"]),
                 masked=rng.choice([0.0, 0.15]))
        if kind == "gate":
            c.update(renorm=rng.random() < 0.6, bias=c["score"] == "sigmoid" and rng.random() < 0.7,
                     backward=rng.random() < 0.7)
        else:
            c.update(S=min(T, _log_int(rng, 1, 64)))
        return c
    if kind == "weights":
        return dict(kind=kind, E=_log_int(rng, 1, 32), N=_log_int(rng, 64, 4096), K=_log_int(rng, 64, 2048),
                    dtype=rng.choice(["bf16", "f32"]))
    while True:
        c = dict(kind=kind, R=_log_int(rng, 1, 32768), N=_log_int(rng, 64, 4096), K=_log_int(rng, 128, 7168),
                 E=_log_int(rng, 1, 64), skew=rng.choice([0.0, 0.6, 1.2]))
        if kind == "product":
            c["K"] = max(128, c["K"] // 128 * 128)
        else:
            c["dtype"] = rng.choice(["bf16", "bf16", "f32"])
        if c["E"] * c["N"] * c["K"] <= 1 << 29 and c["R"] * c["N"] * c["K"] <= 1 << 39:
            return c


def _up(n, m):
    return (n + m - 1) // m * m


def work(case):
    k = case["kind"]
    if k in ("gate", "balance"):
        T, E, K = case["T"], case["E"], case["K"]
        b = 4 if case["dtype"] == "f32" else 2
        if k == "gate":
            nbytes, flops = T * E * b + T * K * 12, 8 * T * E
            if case["backward"]:
                nbytes, flops = nbytes + T * E * b * 2 + T * K * 12, 2 * flops
        else:
            nbytes, flops = T * E * b * 3 + 2 * T * K * 8 + case["S"] * E * 12, 16 * T * E
        return {"bytes": nbytes, "flops": flops}
    E, N, K = case["E"], case["N"], case["K"]
    Kp = _up(K, 128)
    xb = 4 if case.get("dtype") == "f32" else 2
    if k == "weights":
        return {"bytes": E * N * K * xb + E * N * Kp + E * K * _up(N, 128), "flops": 4 * E * N * K}
    R = case["R"]
    used = min(E, R)
    if k == "product":
        return {"bytes": R * Kp + used * N * Kp + R * Kp // 32 + 2 * R * N, "flops": 2 * R * N * Kp}
    if k == "linear":
        return {"bytes": R * K * xb + used * N * Kp + 2 * R * N, "flops": 2 * R * N * K}
    return {"bytes": R * K * xb + R * N * xb + used * N * Kp + 2 * R * K + 2 * E * N * K, "flops": 4 * R * N * K}


# ---- inputs ---------------------------------------------------------------------------------------

def _sizes(case, seed):
    """Rows of each expert: a multinomial draw over a Zipf popularity (skew 0: uniform)."""
    rng = np.random.default_rng(seed)
    p = np.arange(1, case["E"] + 1, dtype=np.float64) ** -case["skew"]
    return rng.multinomial(case["R"], rng.permutation(p / p.sum())).tolist()


def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV) * std


def _activations(g, rows, cols, dtype):
    """Rows of unequal size with a few large channels, as activations have them."""
    x = _normal(g, (rows, cols)) * torch.exp(0.5 * _normal(g, (rows, 1))) * torch.exp(0.7 * _normal(g, (1, cols)))
    return x.to(torch.bfloat16) if dtype == "bf16" else x


def _logits(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    T, E = case["T"], case["E"]
    l = _normal(g, (T, E), 1.3) + _normal(g, (1, E), 0.4)
    l = l.to(torch.bfloat16) if case["dtype"] == "bf16" else l
    mask = (torch.rand(T, generator=g, device=DEV) >= case["masked"]).to(torch.uint8) if case["masked"] else None
    return g, l, mask


def _offsets(sizes):
    return torch.tensor(np.concatenate([[0], np.cumsum(sizes)]), dtype=torch.int32, device=DEV)


def prepare(case, seed):
    k = case["kind"]
    s = dict(case=case)
    if k in ("gate", "balance"):
        T, E, K = case["T"], case["E"], case["K"]
        g, l, mask = _logits(case, seed)
        s.update(logits=l, mask=mask, dlogits=torch.empty_like(l))
        if k == "gate":
            s["bias"] = _normal(g, (E,), 0.05) if case["bias"] else None
            s["dw"] = _normal(g, (T, K))
            s["idx"] = torch.empty((T, K), dtype=torch.int64, device=DEV)
            s["w"] = torch.empty((T, K), dtype=torch.float32, device=DEV)
            return s
        S = case["S"]
        cuts = np.sort(np.random.default_rng(seed).integers(0, T + 1, S - 1)).tolist()
        s["seq"] = torch.tensor([0, *cuts, T], dtype=torch.int32, device=DEV)
        s["idx"] = torch.argsort(l.float(), dim=1, descending=True, stable=True)[:, :K].contiguous()
        if mask is not None:
            s["idx"][mask == 0] = -1
        s["coef"], s["dloss"] = 0.01, torch.full((1,), 1.7, device=DEV)
        s["loss"] = torch.empty(1, device=DEV)
        s["counts"] = torch.empty((S, E), dtype=torch.int32, device=DEV)
        s["slope"] = torch.empty((S, E), device=DEV)
        s["workspace"] = torch.empty(4096 + 8 * E * (T // 16 + 2 * S + 64), dtype=torch.uint8, device=DEV)
        return s
    g = torch.Generator(device=DEV).manual_seed(seed)
    E, N, K = case["E"], case["N"], case["K"]
    Kp, Np = _up(K, 128), _up(N, 128)
    if k == "weights":
        w = _normal(g, (E, N, K), 0.02)
        s["w"] = w.to(torch.bfloat16) if case["dtype"] == "bf16" else w
        s["codes"], s["codes_t"] = _bytes(E, N, Kp), _bytes(E, K, Np)
        s["scales"], s["scales_t"] = _floats(E, Np // 128, Kp // 128), _floats(E, Kp // 128, Np // 128)
        return s
    R = case["R"]
    s["sizes"] = _sizes(case, seed)
    s["offsets"] = _offsets(s["sizes"])
    # the weights as a program keeps them: codes and a scale per 128 x 128
    back = k == "gradients"
    rows, cols = (K, N) if back else (N, K)
    s["w"] = torch.empty((E, rows, _up(cols, 128)), dtype=torch.uint8, device=DEV)
    s["ws"] = torch.empty((E, _up(rows, 128) // 128, _up(cols, 128) // 128), device=DEV)
    for e in range(E):
        c, z = _plain_weights(_normal(g, (1, rows, cols), 0.02))
        s["w"][e], s["ws"][e] = c[0], z[0]
    if k == "product":
        s["a"], s["as"] = _plain_rows(_activations(g, R, K, "bf16"))
        s["out"] = torch.empty((R, N), dtype=torch.bfloat16, device=DEV)
    elif k == "linear":
        s["x"] = _activations(g, R, K, case["dtype"])
        s["a"], s["as"] = _bytes(R, Kp), _floats(Kp // 128, R)
        s["out"] = torch.empty((R, N), dtype=torch.bfloat16, device=DEV)
    else:
        s["x"] = _activations(g, R, K, case["dtype"])
        dy = _activations(g, R, N, "f32") * 1e-3
        s["dy"] = dy.to(torch.bfloat16) if case["dtype"] == "bf16" else dy
        Rp = (R + 127 * E) // 128 * 128
        s["g"], s["gs"] = _bytes(R, Np), _floats(Np // 128, R)
        s["gt"], s["gts"] = _bytes(N, Rp), _bytes(Rp // 128, N)
        s["xt"], s["xts"] = _bytes(K, Rp), _bytes(Rp // 128, K)
        s["dx"] = torch.empty((R, K), dtype=torch.bfloat16, device=DEV)
        s["dw"] = torch.empty((E, N, K), dtype=torch.bfloat16, device=DEV)
    return s


def _bytes(*shape):
    return torch.empty(shape, dtype=torch.uint8, device=DEV)


def _floats(*shape):
    return torch.empty(shape, dtype=torch.float32, device=DEV)


# ---- plain forms ----------------------------------------------------------------------------------

def _pad(x, rows, cols):
    return torch.nn.functional.pad(x, (0, cols - x.shape[-1], 0, rows - x.shape[-2]))


def _plain_rows(x):
    """x [R][C] -> codes [R][Cp], scales [Cp/128][R]: a scale per row and 128 columns."""
    R, C = x.shape
    v = _pad(x.float(), R, _up(C, 128)).view(R, -1, 128)
    scale = torch.clamp_min(v.abs().amax(2) / 448.0, F32_MIN_NORMAL)
    codes = (v * (1.0 / scale)[:, :, None]).to(E4M3)
    return codes.view(torch.uint8).view(R, -1), scale.t().contiguous()


def _plain_weights(w):
    """w [E][N][K] -> codes [E][N][Kp], scales [E][Np/128][Kp/128]."""
    E, N, K = w.shape
    v = _pad(w.float(), _up(N, 128), _up(K, 128))
    v = v.view(E, v.shape[1] // 128, 128, v.shape[2] // 128, 128)
    scale = torch.clamp_min(v.abs().amax((2, 4)) / 448.0, F32_MIN_NORMAL)
    codes = (v * (1.0 / scale)[:, :, None, :, None]).to(E4M3).view(torch.uint8)
    return codes.reshape(E, _up(N, 128), -1)[:, :N].contiguous(), scale


def _plain_columns(x):
    """x [n][C] -> the values of its e4m3 codes, a power-of-two scale per 128 rows of a column."""
    n, C = x.shape
    v = _pad(x.float(), _up(n, 128), C).view(-1, 128, C)
    m, e = torch.frexp(v.abs().amax(1))
    e = torch.clamp_min(e - 9 + (m > 0.875).to(e.dtype), -126)[:, None, :]
    codes = (v * _power_of_two(-e)).to(E4M3)
    return (codes.float() * _power_of_two(e)).view(-1, C)


def _power_of_two(e):
    """2^e in float32, -126 <= e <= 127, by its exponent field (torch.ldexp goes through pow)."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _values(codes, scales):
    """Rows' values: codes [R][Kp], scales [Kp/128][R]."""
    R = codes.shape[0]
    return (codes.view(E4M3).float().view(R, -1, 128) * scales.t()[:, :, None]).view(R, -1)


def _weight_values(codes, scales):
    N, Kp = codes.shape
    return codes.view(E4M3).float() * scales.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)


def _plain_product(s, a, scales, out):
    at = 0
    for e, n in enumerate(s["sizes"]):
        if n:
            v = _values(a[at:at + n], scales[:, at:at + n])
            out[at:at + n] = v @ _weight_values(s["w"][e], s["ws"][e]).t()
        at += n
    return out


def _plain_scores(case, l):
    if case["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    z = torch.exp(l - l.amax(1, keepdim=True))
    return z / z.sum(1, keepdim=True)


def _plain_gate(s):
    c, l = s["case"], s["logits"].float()
    key = l
    if c["score"] == "sigmoid":  # values next to each other decide which expert is chosen: 64 bits
        key = 1.0 / (1.0 + torch.exp(-l.double()))
        key = key + s["bias"].double() if s["bias"] is not None else key
    idx = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :c["K"]]
    p = _plain_scores(c, l)
    sel = p.gather(1, idx)
    total = sel.sum(1, keepdim=True)
    q = sel / total if c["renorm"] else sel
    live = torch.ones_like(idx[:, :1], dtype=torch.bool) if s["mask"] is None else s["mask"][:, None] != 0
    out = [torch.where(live, idx, -1), torch.where(live, q, 0.0)]
    if c["backward"]:
        g = s["dw"]
        if c["renorm"]:
            g = g - (g * q).sum(1, keepdim=True)
            g = q * g if c["score"] == "softmax" else g / total * sel * (1 - sel)
            d = torch.zeros_like(l).scatter_add(1, idx, g)
        elif c["score"] == "sigmoid":
            d = torch.zeros_like(l).scatter_add(1, idx, g * sel * (1 - sel))
        else:
            d = p * (torch.zeros_like(l).scatter_add(1, idx, g) - (g * sel).sum(1, keepdim=True))
        out.append(torch.where(live, d, 0.0).to(s["logits"].dtype))
    return out


def _plain_balance(s):
    c, l = s["case"], s["logits"].float()
    T, E, S = c["T"], c["E"], c["S"]
    seq = torch.searchsorted(s["seq"][1:], torch.arange(T, dtype=torch.int32, device=DEV), right=True)
    live = torch.ones(T, device=DEV, dtype=torch.bool) if s["mask"] is None else s["mask"] != 0
    z = _plain_scores(c, l)
    total = z.sum(1, keepdim=True)
    p = z / total * live[:, None]
    hit = (seq[:, None] * E + s["idx"])[s["idx"] >= 0]
    counts = torch.bincount(hit, minlength=S * E).view(S, E)
    member = (seq[None, :] == torch.arange(S, device=DEV)[:, None]).double()  # [S][T]
    n, sums = (member * live).sum(1), member @ p.double()
    used = (n > 0).sum()
    slope = _over(s["coef"] * E * counts.double(), counts.sum(1, keepdim=True) * n[:, None] * used)
    loss = (slope * sums).sum().float().view(1)
    f = slope.float()[seq] * (s["dloss"] * live[:, None])
    if c["score"] == "softmax":
        d = p * (f - (f * p).sum(1, keepdim=True))
    else:
        d = (f - (f * p).sum(1, keepdim=True)) / total * z * (1 - z)
    return [loss, counts.to(torch.int32), slope.float(), d.to(l.dtype if c["dtype"] == "f32" else torch.bfloat16)]


def _over(a, b):
    """a / b, and 0 where b is 0."""
    return torch.where(b == 0, torch.zeros_like(a), a / torch.where(b == 0, torch.ones_like(a), b))


def _plain_gradients(s):
    g, gs = _plain_rows(s["dy"])
    _plain_product(s, g, gs, s["dx"])
    at = 0
    for e, n in enumerate(s["sizes"]):
        s["dw"][e] = _plain_columns(s["dy"][at:at + n]).t() @ _plain_columns(s["x"][at:at + n])
        at += n
    return [s["dx"], s["dw"]]


def _plain(s):
    k = s["case"]["kind"]
    if k == "gate":
        return _plain_gate(s)
    if k == "balance":
        return _plain_balance(s)
    if k == "weights":
        codes, scales = _plain_weights(s["w"])
        E, N, K = s["w"].shape
        codes_t = _pad(codes[:, :, :K].transpose(1, 2), K, _up(N, 128)).contiguous()
        return [codes.view(E4M3), scales, codes_t.view(E4M3), scales.transpose(1, 2).contiguous()]
    if k == "gradients":
        return _plain_gradients(s)
    a, scales = _plain_rows(s["x"]) if k == "linear" else (s["a"], s["as"])
    return _plain_product(s, a, scales, s["out"])


# ---- the framework's calls ------------------------------------------------------------------------

def _framework(s):
    import combine_dispatch_amd as moe
    c = s["case"]
    k = c["kind"]
    if k == "gate":
        o = moe.gate_options(score=c["score"], renormalise=c["renorm"])
        moe.moe_gate(s["logits"], s["idx"], s["w"], bias=s["bias"], token_mask=s["mask"], opts=o)
        if not c["backward"]:
            return [s["idx"], s["w"]]
        moe.moe_gate_backward(s["logits"], s["dlogits"], topk_idx=s["idx"], d_topk_w=s["dw"], token_mask=s["mask"], opts=o)
        return [s["idx"], s["w"], s["dlogits"]]
    if k == "balance":
        o = moe.gate_options(score=c["score"])
        moe.moe_balance_loss(s["logits"], s["idx"], s["coef"], s["loss"], s["counts"], s["slope"], s["workspace"],
                             seq_offsets=s["seq"], token_mask=s["mask"], opts=o)
        moe.moe_gate_backward(s["logits"], s["dlogits"], slope=s["slope"], d_loss=s["dloss"], seq_offsets=s["seq"],
                              token_mask=s["mask"], opts=o)
        return [s["loss"], s["counts"], s["slope"], s["dlogits"]]
    if k == "weights":
        moe.moe_quantise_weights(s["w"], s["codes"], s["scales"], codes_t=s["codes_t"], scales_t=s["scales_t"])
        return [s["codes"].view(E4M3), s["scales"], s["codes_t"].view(E4M3), s["scales_t"]]
    if k == "gradients":
        moe.moe_quantise_rows(s["dy"], s["g"], s["gs"])
        moe.moe_block_gemm(s["g"], s["gs"], s["w"], s["ws"], s["dx"], offsets=s["offsets"])
        moe.moe_quantise_columns(s["dy"], s["gt"], s["gts"], offsets=s["offsets"])
        moe.moe_quantise_columns(s["x"], s["xt"], s["xts"], offsets=s["offsets"])
        moe.moe_block_gemm_wgrad(s["gt"], s["gts"], s["xt"], s["xts"], s["dw"], rows=c["R"], offsets=s["offsets"])
        return [s["dx"], s["dw"]]
    if k == "linear":
        moe.moe_quantise_rows(s["x"], s["a"], s["as"])
    moe.moe_block_gemm(s["a"], s["as"], s["w"], s["ws"], s["out"], offsets=s["offsets"])
    return s["out"]


def run(state):
    return _framework(state) if own else _plain(state)


# ---- from the definitions, in 64 bits --------------------------------------------------------------

def _power_of_two64(e):
    return ((e.long() + 1023) << 52).view(torch.float64)


def _round_e4m3(v):
    """The nearest e4m3 value, halves to even, of |v| <= 448."""
    e = torch.clamp_min(torch.frexp(v)[1] - 1, -6)
    step = _power_of_two64(e - 3)
    return torch.clamp(torch.round(v / step) * step, -448.0, 448.0)


def _blocks64(v, dims, power_of_two=False):
    """The values that v's e4m3 blocks stand for: blocks of 128 along `dims`. Also codes' values and scales."""
    shape = v.shape
    want = [_up(n, 128) if d in dims else n for d, n in enumerate(shape)]
    p = torch.zeros(want, dtype=torch.float64, device=v.device)
    p[tuple(slice(0, n) for n in shape)] = v
    split, over = [], []
    for d, n in enumerate(want):
        if d in dims:
            split += [n // 128, 128]
            over.append(len(split) - 1)
        else:
            split.append(n)
    p = p.view(split)
    scale = p.abs().amax(over, keepdim=True) / 448.0
    if power_of_two:
        m, e = torch.frexp(torch.clamp_min(scale, F32_MIN_NORMAL))
        scale = _power_of_two64(torch.where(m == 0.5, e - 1, e))  # the smallest one that is not less
    else:
        scale = torch.clamp_min(scale, F32_MIN_NORMAL)
    q = _round_e4m3(p / scale)
    cut = tuple(slice(0, n) for n in shape)
    return (q * scale).view(want)[cut], q.view(want), scale.squeeze(over)


def _decode64(codes):
    """e4m3 bytes -> values, by their fields."""
    c = codes.to(torch.int32)
    e, m = (c >> 3) & 15, (c & 7).double()
    v = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * _power_of_two64(e - 7))
    return torch.where(c >= 128, -v, v)


def _weights64(s, e, rows, cols):
    w = _decode64(s["w"][e])
    n, k = torch.arange(w.shape[0], device=DEV) // 128, torch.arange(w.shape[1], device=DEV) // 128
    return (w * s["ws"][e].double()[n][:, k])[:rows, :cols]


def _groups(s):
    at = 0
    for e, n in enumerate(s["sizes"]):
        yield e, at, at + n
        at += n


def exact(case, seed):
    s = prepare(case, seed)
    k = case["kind"]
    if k == "gate":
        return _exact_gate(s)
    if k == "balance":
        return _exact_balance(s)
    if k == "weights":
        v, q, scale = _blocks64(s["w"].double(), (1, 2))
        N, K = case["N"], case["K"]
        qt = q.transpose(1, 2)[:, :K].contiguous()
        return [q[:, :N].contiguous(), scale, qt, scale.transpose(1, 2).contiguous()]
    N, K = case["N"], case["K"]
    if k == "gradients":
        dx = torch.zeros((case["R"], K), dtype=torch.float64, device=DEV)
        dw = torch.zeros((case["E"], N, K), dtype=torch.float64, device=DEV)
        for e, lo, hi in _groups(s):
            dy, x = s["dy"][lo:hi].double(), s["x"][lo:hi].double()
            if hi > lo:
                dx[lo:hi] = _blocks64(dy, (1,))[0] @ _weights64(s, e, K, N).t().contiguous()
                dw[e] = _blocks64(dy, (0,), True)[0].t().contiguous() @ _blocks64(x, (0,), True)[0]
        return [dx, dw]
    out = torch.zeros((case["R"], N), dtype=torch.float64, device=DEV)
    for e, lo, hi in _groups(s):
        if hi == lo:
            continue
        if k == "linear":
            v = _blocks64(s["x"][lo:hi].double(), (1,))[0]
        else:
            kb = torch.arange(K, device=DEV) // 128
            v = _decode64(s["a"][lo:hi]) * s["as"][:, lo:hi].double().t()[:, kb]
        out[lo:hi] = v @ _weights64(s, e, N, K).t().contiguous()
    return out


def _softmax64(l):
    return torch.exp(l - torch.logsumexp(l, 1, keepdim=True))


def _exact_gate(s):
    c, l = s["case"], s["logits"].double()
    sig = c["score"] == "sigmoid"
    score = torch.sigmoid(l) if sig else _softmax64(l)
    key = l if not sig else score + (0.0 if s["bias"] is None else s["bias"].double())
    chosen = torch.argsort(-key, dim=1, stable=True)[:, :c["K"]]
    dead = torch.zeros(c["T"], dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"] == 0
    # weights and the gradient by autograd of the definition
    leaf = l.clone().requires_grad_()
    sc = torch.sigmoid(leaf) if sig else torch.softmax(leaf, 1)
    w = sc.gather(1, chosen)
    w = w / w.sum(1, keepdim=True) if c["renorm"] else w
    (d,) = torch.autograd.grad(w, leaf, s["dw"].double().masked_fill(dead[:, None], 0.0))
    out = [chosen.masked_fill(dead[:, None], -1), w.detach().masked_fill(dead[:, None], 0.0)]
    return out + [d] if c["backward"] else out


def _exact_balance(s):
    c, l = s["case"], s["logits"].double().requires_grad_()
    S, E = c["S"], c["E"]
    z = torch.sigmoid(l) if c["score"] == "sigmoid" else torch.softmax(l, 1)
    p = z / z.sum(1, keepdim=True)
    live = torch.ones(c["T"], dtype=torch.float64, device=DEV) if s["mask"] is None else (s["mask"] != 0).double()
    bounds = s["seq"].tolist()
    counts = torch.zeros((S, E), dtype=torch.int32, device=DEV)
    slope = torch.zeros((S, E), dtype=torch.float64, device=DEV)
    loss = torch.zeros((), dtype=torch.float64, device=DEV)
    lens = [float(live[a:b].sum()) for a, b in zip(bounds, bounds[1:])]
    used = sum(n > 0 for n in lens)
    for q, (a, b) in enumerate(zip(bounds, bounds[1:])):
        i = s["idx"][a:b]
        counts[q] = torch.bincount(i[i >= 0], minlength=E).to(torch.int32)
        if lens[q] and int(counts[q].sum()):
            f = counts[q].double() * E / counts[q].sum().double()
            slope[q] = s["coef"] * f / (used * lens[q])
            loss = loss + s["coef"] / used * (f * (p[a:b] * live[a:b, None]).sum(0) / lens[q]).sum()
    (d,) = torch.autograd.grad(loss, l, s["dloss"].double()[0])
    return [loss.detach().view(1), counts, slope, d]
