"""Measured cases of the operators around the block-scaled products.

Three operators, each in a plain form (elementary torch operations) and, where
``own`` is true, as the calls a user makes of ``hadamard_rotated_bit_gb300``:

``norm``   h = x + residual (rounded to the residual's type), the root-mean-square
           norm n = h / sqrt(mean(h^2) + eps) * w, and n rotated and quantized for the
           next product: integer codes (one or two FP8 bytes each) and one fp32
           scale per 32 values, block-major.
``route``  router scores (softmax or sigmoid of the logits), keys = scores + bias,
           the best groups of experts by their best keys, the k experts of largest
           key in them, their weights, and the rows grouped by expert.
``gemm``   the block-scaled product z = X W^T of Q4_0 weights (one FP8 byte per code,
           fp32 scale per 32) with 4- or 8-bit activations, then
           y = act(z + bias) + residual; "swiglu" takes interleaved gate and up rows
           and gives silu(gate) * up.

Quantized outputs come as FP8 views: each byte as the number it stands for.
"""
import math

import numpy as np
import torch

own = False

F8, F8W = torch.float8_e4m3fn, torch.float8_e5m2
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HIDDEN, FFN = 5120, 17408             # the dense chain's widths
MOE_HIDDEN, MOE_E, MOE_K = 2048, 128, 8   # the expert layer's


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _norm(name, M, K, x, res, form, rotate, norm_out=""):
    return {"name": name, "op": "norm", "M": M, "K": K, "x": x, "res": res, "form": form,
            "rotate": rotate, "norm_out": norm_out, "eps": 1e-6}


def _route(name, T, E, k, score, bias, n_group, topk_group, group_top, renorm, scale):
    return {"name": name, "op": "route", "T": T, "E": E, "k": k, "score": score, "bias": bias,
            "n_group": n_group, "topk_group": topk_group, "group_top": group_top,
            "renorm": renorm, "scale": scale}


def _gemm(name, M, N, K, bits, bias, act, res, y):
    return {"name": name, "op": "gemm", "M": M, "N": N, "K": K, "bits": bits, "bias": bias,
            "act": act, "res": res, "y": y}


def listed():
    return [
        # one new token between two layers: the attention product's fp32 output added to
        # the bf16 residual stream, normed and quantized for gate/up
        _norm("norm token", 1, HIDDEN, "f32", "bf16", "q4_tc", 32),
        # the same for the 512-token prompt of the dense chain
        _norm("norm prompt", 512, HIDDEN, "f32", "bf16", "q4_tc", 32),
        # in front of an expert layer: fp32 residual stream, 8-bit codes, and the normed
        # rows themselves in bf16 (the router's and the gathering quantizer's input)
        _norm("norm expert layer", 1024, MOE_HIDDEN, "bf16", "f32", "q8_tc", 64, "bf16"),
        # a long prompt taken as one batch, everything in bf16
        _norm("norm long prompt", 16384, HIDDEN, "bf16", "bf16", "q4_tc", 32),
        # one new token through the router of the expert layer
        _route("route token", 1, MOE_E, MOE_K, "softmax", False, 1, 1, 1, True, 1.0),
        # its 1024-token micro-batch, with a balance bias on the keys
        _route("route micro-batch", 1024, MOE_E, MOE_K, "softmax", True, 1, 1, 1, True, 1.0),
        # a ragged batch with groups by their best expert, weights not renormalised
        _route("route ragged groups", 777, 160, 6, "softmax", False, 8, 3, 1, False, 16.0),
        # a long batch with sigmoid scores, bias, groups by their two best experts
        _route("route long", 16384, 256, 8, "sigmoid", True, 8, 4, 2, True, 2.5),
        # one new token through the attention output projection, added to the residual
        _gemm("gemm token", 1, HIDDEN, HIDDEN, 4, False, "none", "f32", "f32"),
        # a handful of sequences, one token each, through gate/up with its activation
        _gemm("gemm few tokens", 5, 2 * FFN, HIDDEN, 4, False, "swiglu", "", "bf16"),
        # a ragged prompt through FFN down on the exact 8-bit route, with the residual
        _gemm("gemm down 8-bit", 333, HIDDEN, FFN, 8, True, "none", "bf16", "bf16"),
        # the 512-token prompt through gate/up with its activation: the largest product
        _gemm("gemm gate/up", 512, 2 * FFN, HIDDEN, 4, False, "swiglu", "", "bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("norm", "route", "gemm"))
    if op == "norm":
        rotate = rng.choice((0, 32, 64, 128))
        step = max(32, rotate)
        K = step * max(1, _log(rng, 256, FFN) // step)
        M = min(_log(rng, 1, 16384), 16384 * HIDDEN // (2 * K))
        c = _norm("", M, K, rng.choice(("bf16", "f32")), rng.choice(("", "bf16", "f32")),
                  rng.choice(("q4_tc", "q8_tc", "q4_tc_e5m2")), rotate,
                  rng.choice(("", "", "bf16", "f32")))
    elif op == "route":
        n_group = rng.choice((1, 1, 2, 4, 8, 5))
        size = max(2, _log(rng, 16, 512) // n_group)
        E = size * n_group
        topk_group = rng.randint(1, n_group)
        k = min(rng.randint(1, 12), topk_group * size)
        T = min(_log(rng, 1, 16384), 16384 * 256 // E)
        c = _route("", T, E, k, rng.choice(("softmax", "sigmoid")), rng.random() < 0.6, n_group,
                   topk_group, rng.choice((1, 2)), rng.random() < 0.7, rng.choice((1.0, 2.5)))
    else:
        K = 128 * max(1, _log(rng, 256, FFN) // 128)
        N = 32 * max(1, _log(rng, 64, 2 * FFN) // 32)
        M = _log(rng, 1, 512)
        while M * N * K > 512 * 2 * FFN * HIDDEN:
            M = max(1, M // 2)
        c = _gemm("", M, N, K, rng.choice((4, 4, 8)), rng.random() < 0.5,
                  rng.choice(("none", "relu", "silu", "gelu_tanh", "gelu_erf", "swiglu")),
                  rng.choice(("", "bf16", "f32")), rng.choice(("bf16", "f32")))
    del c["name"]
    return c


# ----------------------------------------------------------------------------
# what a user's program has in hand
# ----------------------------------------------------------------------------
def _act_rows(M, K, g):
    """N(0, 1) rows with 0.5% of the channels 30 times larger."""
    x = torch.randn((M, K), device="cuda", generator=g)
    n = max(1, round(0.005 * K))
    x[:, torch.randperm(K, device="cuda", generator=g)[:n]] *= 30.0
    return x


def _signs(n):
    """Sylvester's n x n matrix of signs: (-1)^popcount(i & j)."""
    i = torch.arange(n, device="cuda")   # n <= 128: seven bits to fold
    b = i[:, None] & i[None, :]
    b = b ^ (b >> 4)
    b = b ^ (b >> 2)
    b = (b ^ (b >> 1)) & 1
    return (1 - 2 * b).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    if c["op"] == "norm":
        M, K = c["M"], c["K"]
        c["x_t"] = _act_rows(M, K, g).to(DT[c["x"]])
        c["res_t"] = (2.0 * _act_rows(M, K, g)).to(DT[c["res"]]) if c["res"] else None
        c["w_t"] = 1.0 + 0.1 * torch.randn(K, device="cuda", generator=g)
        c["signs"] = _signs(c["rotate"]) if c["rotate"] else None
    elif c["op"] == "route":
        c["logits"] = 1.5 * torch.randn((c["T"], c["E"]), device="cuda", generator=g)
        c["bias_t"] = 0.02 * torch.randn(c["E"], device="cuda", generator=g) if c["bias"] else None
    else:
        M, N, K = c["M"], c["N"], c["K"]
        nb = K // 32
        # Q4_0 weights: the value of largest magnitude maps to -8, fp16 scales
        w = (0.02 * torch.randn((N, nb, 32), device="cuda", generator=g))
        d = w.gather(2, w.abs().argmax(2, keepdim=True)) / -8.0
        q = torch.clamp(torch.floor(w / d + 8.5), 0, 15) - 8.0
        c["wp"] = q.reshape(N, K).to(F8).view(torch.uint8)
        c["wsc"] = torch.zeros((N, (nb + 3) // 4 * 4), device="cuda")
        c["wsc"][:, :nb] = d.reshape(N, nb).half().float()
        del w, d, q
        # activations: 4- or 8-bit codes of spread rows, scales block-major
        x = torch.randn((M, nb, 32), device="cuda", generator=g)
        top = 7.0 if c["bits"] == 4 else 127.0
        d = x.abs().amax(2, keepdim=True) / top
        q = torch.round(x / d)
        if c["bits"] == 8:
            h = torch.floor(q / 16.0)
            q = torch.cat((16.0 * h, q - 16.0 * h), 2)
        c["xw"] = q.reshape(M, -1).to(F8).view(torch.uint8)
        c["xdt"] = torch.zeros((nb, (M + 3) // 4 * 4), device="cuda")
        c["xdt"][:, :M] = d.reshape(M, nb).t()
        c["bias_t"] = 0.1 * torch.randn(N, device="cuda", generator=g) if c["bias"] else None
        n_out = N // 2 if c["act"] == "swiglu" else N
        c["res_t"] = (torch.randn((M, n_out), device="cuda", generator=g).to(DT[c["res"]])
                      if c["res"] else None)
    return c


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(state):
    return _RUN[state["op"]](state)


def _run_norm(s):
    if own:
        import hadamard_rotated_bit_gb300 as h32
        xw, xd, res, nrm = h32.h32_add_rms_norm_quantize(
            s["x_t"], s["w_t"], residual=s["res_t"], eps=s["eps"], form=s["form"],
            rotate=s["rotate"], norm_out=DT[s["norm_out"]] if s["norm_out"] else None)
        return {"codes": xw.view(F8W if s["form"] == "q4_tc_e5m2" else F8),
                "scales": xd[:, :s["M"]], "residual": res, "norm": nrm}
    M, K = s["x_t"].shape
    h = s["x_t"].float()
    res = None
    if s["res_t"] is not None:
        res = (h + s["res_t"].float()).to(s["res_t"].dtype)
        h = res.float()
    # the mean in 64 bits: codes next to a rounding border follow from it
    ms = (h.double().square().mean(1, keepdim=True) + s["eps"]).float()
    n = h * (1.0 / torch.sqrt(ms)) * s["w_t"]
    nrm = n.to(DT[s["norm_out"]]) if s["norm_out"] else None
    v = n
    if s["rotate"]:
        r = s["rotate"]
        v = (v.reshape(-1, r) @ s["signs"]) * (1.0 / math.sqrt(r))
    v = v.reshape(M, K // 32, 32)
    top = 127.0 if s["form"] == "q8_tc" else 7.0
    d = v.abs().amax(2, keepdim=True) / top
    q = torch.round(v * torch.where(d > 0, 1.0 / d, 0.0))
    if s["form"] == "q8_tc":
        hi = torch.floor(q / 16.0)
        codes = torch.cat((16.0 * hi, q - 16.0 * hi), 2).reshape(M, 2 * K).to(F8)
    elif s["form"] == "q4_tc":
        codes = q.reshape(M, K).to(F8)
    else:
        codes = (512.0 * q).reshape(M, K).to(F8W)
    return {"codes": codes, "scales": d.reshape(M, K // 32).t().contiguous(), "residual": res,
            "norm": nrm}


def _run_route(s):
    if own:
        import hadamard_rotated_bit_gb300 as h32
        ids, w, off, row_idx, row_of = h32.h32_moe_route_scored(
            s["logits"], s["k"], score=s["score"], bias=s["bias_t"], n_group=s["n_group"],
            topk_group=s["topk_group"], group_top=s["group_top"], renormalize=s["renorm"],
            scale=s["scale"])
        return {"ids": ids, "weights": w, "offsets": off, "row_idx": row_idx, "row_of": row_of}
    T, E = s["logits"].shape
    k, G = s["k"], s["n_group"]
    l = s["logits"].double()   # near ties are decided in 64 bits
    if s["score"] == "sigmoid":
        sc = 1.0 / (1.0 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(1, keepdim=True))
        sc = e / e.sum(1, keepdim=True)
    key = sc if s["bias_t"] is None else sc + s["bias_t"].double()
    if G > 1:
        best = torch.sort(key.reshape(T, G, E // G), dim=2, descending=True).values
        gs = best[:, :, :s["group_top"]].sum(2)
        groups = torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :s["topk_group"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, groups, True)
        key = torch.where(keep.repeat_interleave(E // G, 1), key, -math.inf)
    ids = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
    w = sc.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    w = (w * s["scale"]).float()
    flat = ids.reshape(-1)
    order = torch.sort(flat, dim=0, stable=True).indices
    row_of = torch.empty_like(order)
    row_of[order] = torch.arange(T * k, device=l.device)
    off = torch.zeros(E + 1, dtype=torch.int64, device=l.device)
    off[1:] = torch.cumsum((flat[:, None] == torch.arange(E, device=l.device)).sum(0), 0)
    i32 = torch.int32
    return {"ids": ids.to(i32), "weights": w, "offsets": off.to(i32), "row_idx": (order // k).to(i32),
            "row_of": row_of.reshape(T, k).to(i32)}


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "gelu_erf":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if act == "swiglu":
        gate, up = z[:, 0::2], z[:, 1::2]
        return gate / (1.0 + torch.exp(-gate)) * up
    return z


def _run_gemm(s):
    if own:
        import hadamard_rotated_bit_gb300 as h32
        call = h32.q4_0_x_q4_gemm_tc_epilogue if s["bits"] == 4 else h32.q4_0_x_q8_gemm_tc_epilogue
        return call(s["wp"], s["wsc"], s["xw"], s["xdt"], bias=s["bias_t"], act=s["act"],
                    residual=s["res_t"], y_dtype=DT[s["y"]])
    N, K = s["wp"].shape
    M, nb = s["xw"].shape[0], K // 32
    w = s["wp"].view(F8).float().reshape(N, nb, 32) * s["wsc"][:, :nb, None]
    x = s["xw"].view(F8).float().reshape(M, nb, -1, 32).sum(2) * s["xdt"][:, :M].t()[:, :, None]
    z = x.reshape(M, K) @ w.reshape(N, K).t()
    if s["bias_t"] is not None:
        z = z + s["bias_t"]
    y = _act(z, s["act"])
    if s["res_t"] is not None:
        y = y + s["res_t"].float()
    return y.to(DT[s["y"]])


_RUN = {"norm": _run_norm, "route": _run_route, "gemm": _run_gemm}


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    c = case
    size = {"": 0, "bf16": 2, "f32": 4}
    if c["op"] == "norm":
        n = c["M"] * c["K"]
        code = 2 if c["form"] == "q8_tc" else 1
        turn = int(math.log2(c["rotate"])) + 1 if c["rotate"] else 0
        return {"bytes": n * (size[c["x"]] + 2 * size[c["res"]] + size[c["norm_out"]] + code)
                + n // 32 * 4 + 4 * c["K"], "flops": n * (8 + turn)}
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": 4 * T * E + (4 * E if c["bias"] else 0) + 16 * T * k + 4 * (E + 1),
                "flops": T * E * 4 + T * k * 4}
    M, N, K = c["M"], c["N"], c["K"]
    n_out = N // 2 if c["act"] == "swiglu" else N
    return {"bytes": N * K + N * K // 8 + M * K * (c["bits"] // 4) + M * K // 8
            + M * n_out * (size[c["res"]] + size[c["y"]]) + (4 * N if c["bias"] else 0),
            "flops": 2 * M * N * K}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "route": _exact_route, "gemm": _exact_gemm}[s["op"]](s)


def _exact_norm(s):
    M, K = s["M"], s["K"]
    h = s["x_t"].double()
    res = None
    if s["res_t"] is not None:
        res = h + s["res_t"].double()
        # the norm reads the residual as it is stored
        h = res.float().to(s["res_t"].dtype).double()
    n = h * torch.rsqrt((h * h).sum(1) / K + s["eps"])[:, None] * s["w_t"].double()
    v = n.clone()
    half = 1
    while half < s["rotate"]:   # the butterfly of the transform, stride by stride
        p = v.reshape(M, -1, 2, half)
        v = torch.stack((p[:, :, 0] + p[:, :, 1], p[:, :, 0] - p[:, :, 1]), 2).reshape(M, K)
        half *= 2
    v = v / math.sqrt(s["rotate"] or 1)
    blocks = v.reshape(M, K // 32, 32)
    d = blocks.abs().max(2).values / (127.0 if s["form"] == "q8_tc" else 7.0)
    q = torch.round(blocks / d[:, :, None].clamp_min(1e-300))
    if s["form"] == "q8_tc":
        low = torch.remainder(q, 16.0)
        q = torch.stack((q - low, low), 2)
    elif s["form"] == "q4_tc_e5m2":
        q = q * 512.0
    return {"codes": q.reshape(M, -1), "scales": d.t().contiguous(), "residual": res,
            "norm": n if s["norm_out"] else None}


def _exact_route(s):
    T, E, k, G = s["T"], s["E"], s["k"], s["n_group"]
    l = s["logits"].cpu().numpy().astype(np.float64)
    if s["score"] == "sigmoid":
        sc = np.where(l >= 0, 1.0 / (1.0 + np.exp(-np.abs(l))),
                      np.exp(-np.abs(l)) / (1.0 + np.exp(-np.abs(l))))
    else:
        sc = np.exp(l - np.log(np.exp(l).sum(1, keepdims=True)))
    key = sc.copy()
    if s["bias_t"] is not None:
        key += s["bias_t"].cpu().numpy().astype(np.float64)
    if G > 1:
        by_group = -np.sort(-key.reshape(T, G, -1), axis=2)
        gs = by_group[:, :, :s["group_top"]].sum(2)
        out = np.argsort(-gs, axis=1, kind="stable")[:, s["topk_group"]:]
        masked = key.reshape(T, G, -1)
        np.put_along_axis(masked, out[:, :, None], -np.inf, axis=1)
        key = masked.reshape(T, E)
    ids = np.argsort(-key, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(sc, ids, 1)
    if s["renorm"]:
        w = w / w.sum(1, keepdims=True)
    tok = np.repeat(np.arange(T), k)
    order = np.lexsort((tok, ids.reshape(-1)))
    row_of = np.empty(T * k, np.int32)
    row_of[order] = np.arange(T * k, dtype=np.int32)
    off = np.concatenate(([0], np.cumsum(np.bincount(ids.reshape(-1), minlength=E))))
    return {"ids": ids.astype(np.int32), "weights": w * s["scale"], "offsets": off.astype(np.int32),
            "row_idx": tok[order].astype(np.int32), "row_of": row_of.reshape(T, k)}


def _exact_gemm(s):
    N, K, M = s["N"], s["K"], s["M"]
    w = s["wp"].view(F8).to(torch.float64)
    w *= torch.repeat_interleave(s["wsc"][:, :K // 32].double(), 32, dim=1)
    x = s["xw"].view(F8).to(torch.float64)
    if s["bits"] == 8:
        pair = x.view(M, K // 32, 64)
        x = (pair[:, :, :32] + pair[:, :, 32:]).reshape(M, K)
    x = x * torch.repeat_interleave(s["xdt"][:, :M].double().t(), 32, dim=1)
    z = torch.mm(x, w.t())
    if s["bias_t"] is not None:
        z += s["bias_t"].double()
    a = s["act"]
    if a == "relu":
        z = z.clamp_min(0.0)
    elif a == "silu":
        z = z * torch.sigmoid(z)
    elif a == "gelu_tanh":
        z = z * torch.sigmoid(2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z ** 3))
    elif a == "gelu_erf":
        z = 0.5 * z * torch.special.erfc(-z / math.sqrt(2.0))
    elif a == "swiglu":
        pair = z.view(M, N // 2, 2)
        z = pair[:, :, 0] * torch.sigmoid(pair[:, :, 0]) * pair[:, :, 1]
    if s["res_t"] is not None:
        z = z + s["res_t"].double()
    return z
