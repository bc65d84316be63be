"""Measured cases of the 8-bit floating-point products with a scale for each block of 128,
and of the token log probabilities behind the output head.

Four operators, each in a plain form (elementary torch operations) and, where ``own`` is
true, as the calls a user makes of ``hadamard_rotated_bit_gb300``:

``quant``     activations (groups of 128 of a row, rows gathered by an index where experts
              follow) or weights (blocks of 128 x 128), rotated by a Walsh-Hadamard transform
              of 0, 32, 64 or 128 points, to e4m3 codes and one fp32 scale amax / 448 each.
``product``   y = sum over the blocks of 128 of (d_x d_w) (x_codes . w_codes).
``experts``   the same per expert, over rows grouped by expert.
``logprobs``  log softmax of each row of logits at given tokens, the row's entropy, and its
              k most probable tokens with their log probabilities.

Quantized outputs come as FP8 views: each byte as the number it stands for.
"""
import math

import torch

own = False

F8 = torch.float8_e4m3fn
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
HIDDEN, FFN = 5120, 17408                 # the dense chain's widths
MOE_HIDDEN, MOE_INTER, MOE_E, MOE_K = 2048, 768, 128, 8   # the expert layer's
VOCAB = 131072                            # an output head's rows


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def _quant(name, kind, M, K, x, rotate, R=0):
    return {"name": name, "op": "quant", "kind": kind, "M": M, "K": K, "x": x, "rotate": rotate, "R": R}


def _product(name, M, N, K, y):
    return {"name": name, "op": "product", "M": M, "N": N, "K": K, "y": y}


def _experts(name, T, k, E, N, K, y):
    return {"name": name, "op": "experts", "T": T, "k": k, "E": E, "N": N, "K": K, "y": y}


def _logprobs(name, T, V, x, n, top, masked):
    return {"name": name, "op": "logprobs", "T": T, "V": V, "x": x, "n": n, "top": top, "masked": masked}


def listed():
    return [
        # one new token in front of a product
        _quant("quant token", "act", 1, HIDDEN, "bf16", 128),
        # the expert layer's 1024-token micro-batch: rows gathered in grouped order
        _quant("quant expert rows", "act", 1024, MOE_HIDDEN, "bf16", 0, 1024 * MOE_K),
        # a gate/up projection's weights, once, offline
        _quant("quant weights", "weight", 2 * FFN, HIDDEN, "f32", 128),
        # one new token through the output head: the weights are read once
        _product("product head token", 1, VOCAB, HIDDEN, "f32"),
        # a handful of sequences, one token each, through a square projection
        _product("product few tokens", 7, HIDDEN, HIDDEN, "bf16"),
        # a ragged prompt through FFN down
        _product("product ragged down", 333, HIDDEN, FFN, "f32"),
        # a batch of prompts through gate/up: the largest product
        _product("product gate/up", 4096, 2 * FFN, HIDDEN, "bf16"),
        # 16 sequences' new tokens through the expert layer: a row or two an expert
        _experts("experts tokens", 16, MOE_K, MOE_E, 2 * MOE_INTER, MOE_HIDDEN, "f32"),
        # its 1024-token micro-batch, about 64 rows an expert
        _experts("experts micro-batch", 1024, MOE_K, MOE_E, 2 * MOE_INTER, MOE_HIDDEN, "bf16"),
        # one new token's alternatives
        _logprobs("logprobs token", 1, VOCAB, "f32", 1, 20, False),
        # a scored prompt: odd vocabulary, a third of it masked, one empty row
        _logprobs("logprobs prompt", 512, 100003, "f32", 1, 5, True),
        # a long scored batch, four candidate tokens a row
        _logprobs("logprobs batch", 4096, VOCAB, "bf16", 4, 8, False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("quant", "product", "product", "experts", "logprobs"))
    if op == "quant":
        rotate = rng.choice((0, 32, 64, 128))
        step = max(32, rotate)
        K = step * max(1, _log(rng, 64, FFN) // step)
        if rng.random() < 0.4:
            c = _quant("", "weight", min(_log(rng, 1, 2 * FFN), 2 * FFN * HIDDEN // K), K,
                       rng.choice(("f32", "bf16")), rotate)
        else:
            M = min(_log(rng, 1, 16384), 16384 * HIDDEN // (2 * K))
            R = _log(rng, 1, 4 * M) if rng.random() < 0.4 else 0
            c = _quant("", "act", M, K, rng.choice(("bf16", "f32")), rotate, R)
    elif op == "product":
        K = 32 * max(1, _log(rng, 64, FFN) // 32)
        N = min(_log(rng, 32, VOCAB), VOCAB * HIDDEN // K)
        M = _log(rng, 1, 4096)
        while M * N * K > 4096 * 2 * FFN * HIDDEN:
            M = max(1, M // 2)
        c = _product("", M, N, K, rng.choice(("bf16", "f32")))
    elif op == "experts":
        E = _log(rng, 4, 160)
        c = _experts("", _log(rng, 1, 4096), rng.randint(1, min(8, E)), E, _log(rng, 64, 2048),
                     32 * _log(rng, 4, 80), rng.choice(("bf16", "f32")))
    else:
        V = _log(rng, 1000, VOCAB)
        c = _logprobs("", min(_log(rng, 1, 4096), 4096 * VOCAB // (2 * V)), V,
                      rng.choice(("bf16", "f32")), rng.choice((0, 1, 1, 3)),
                      rng.choice((1, 2, 5, 20, 32)), rng.random() < 0.4)
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


def _blocks(v, rows, cols):
    """v [M][K] as [ceil(M / rows)][rows][ceil(K / cols)][cols], zeros behind the edges."""
    M, K = v.shape
    v = torch.nn.functional.pad(v, (0, -K % cols, 0, -M % rows))
    return v.reshape(v.shape[0] // rows, rows, v.shape[1] // cols, cols)


def _quantize(v, rows):
    """(codes [M][K] e4m3, scales [ceil(M / rows)][ceil(K / 128)]) of blocks of rows x 128."""
    M, K = v.shape
    b = _blocks(v, rows, 128)
    d = b.abs().amax((1, 3), keepdim=True) / 448.0
    q = (b * torch.where(d > 0, 1.0 / d, 0.0)).to(F8)
    return q.reshape(q.shape[0] * rows, -1)[:M, :K].contiguous(), d[:, 0, :, 0].contiguous()


def _code_rows(M, K, g, gain):
    """Codes of N(0, 1) rows, as a quantizer leaves them, and their scales group-major."""
    q, d = _quantize(gain * torch.randn((M, K), device="cuda", generator=g), 1)
    xd = torch.zeros((d.shape[1], (M + 3) // 4 * 4), device="cuda")
    xd[:, :M] = d.t()
    return q.view(torch.uint8), xd


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    c = dict(case)
    if c["op"] == "quant":
        M, K = c["M"], c["K"]
        c["x_t"] = (_act_rows(M, K, g) if c["kind"] == "act"
                    else 0.02 * torch.randn((M, K), device="cuda", generator=g)).to(DT[c["x"]])
        c["signs"] = _signs(c["rotate"]) if c["rotate"] else None
        c["rows"] = (torch.randint(0, M, (c["R"],), device="cuda", generator=g, dtype=torch.int32)
                     if c["R"] else None)
    elif c["op"] == "product":
        wq, c["wd"] = _quantize(0.02 * torch.randn((c["N"], c["K"]), device="cuda", generator=g), 128)
        c["wq"] = wq.view(torch.uint8)
        c["xq"], c["xd"] = _code_rows(c["M"], c["K"], g, 1.0)
    elif c["op"] == "experts":
        T, k, E, N, K = c["T"], c["k"], c["E"], c["N"], c["K"]
        w = 0.02 * torch.randn((E, N, K), device="cuda", generator=g)
        w = torch.nn.functional.pad(w, (0, 0, 0, -N % 128)).reshape(-1, K)
        wq, c["wd"] = _quantize(w, 128)
        c["wq"] = wq.reshape(E, -1, K)[:, :N].reshape(E * N, K).contiguous().view(torch.uint8)
        del w, wq
        ids = torch.rand((T, E), device="cuda", generator=g).argsort(1)[:, :k].reshape(-1)
        count = torch.bincount(ids, minlength=E)
        c["off"] = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        c["off"][1:] = count.cumsum(0)
        c["most"] = int(count.max())
        c["xq"], c["xd"] = _code_rows(T * k, K, g, 1.0)
    else:
        T, V, n = c["T"], c["V"], c["n"]
        # a few likely tokens over a wide floor, as a trained head gives
        l = 2.0 * torch.randn((T, V), device="cuda", generator=g)
        at = torch.randint(0, V, (T, 8), device="cuda", generator=g)
        l.scatter_(1, at, 8.0 + 3.0 * torch.randn((T, 8), device="cuda", generator=g))
        if c["masked"]:
            l[:, torch.rand(V, device="cuda", generator=g) < 0.3] = -math.inf
            if T > 1:
                l[T // 2] = -math.inf    # a row whose mask leaves nothing
        c["logits"] = l.to(DT[c["x"]])
        c["targets"] = None
        if n:
            t = torch.randint(0, V, (T, n), device="cuda", generator=g, dtype=torch.int32)
            t[:, 0] = torch.where(torch.rand(T, device="cuda", generator=g) < 0.7, at[:, 0].int(), t[:, 0])
            t[T - T // 8:] = -1          # rows of padding: no token given
            c["targets"] = t
    return c


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(state):
    return _RUN[state["op"]](state)


def _run_quant(s):
    act = s["kind"] == "act"
    if own:
        import hadamard_rotated_bit_gb300 as h32
        if act:
            q, d = h32.h32_quantize_act_f8(s["x_t"], rotate=s["rotate"], row_idx=s["rows"])
            return {"codes": q.view(F8), "scales": d[:, :q.shape[0]]}
        q, d = h32.h32_quantize_weights_f8(s["x_t"], rotate=s["rotate"])
        return {"codes": q.view(F8), "scales": d}
    v = s["x_t"] if s["rows"] is None else s["x_t"][s["rows"].long()]
    v = v.float()
    if s["rotate"]:
        r = s["rotate"]
        v = ((v.reshape(-1, r) @ s["signs"]) * (1.0 / math.sqrt(r))).reshape(v.shape)
    q, d = _quantize(v, 1 if act else 128)
    return {"codes": q, "scales": d.t().contiguous() if act else d}


def _weights(s):
    """The weights' values [N][K] (fp32: exact products of a code and a scale, rounded once)."""
    N, K = s["wq"].shape
    w = s["wq"].view(F8).float()
    d = s["wd"].repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
    return w * d


def _rows(s):
    M, K = s["xq"].shape
    return s["xq"].view(F8).float() * s["xd"][:, :M].t().repeat_interleave(128, 1)[:, :K]


def _run_product(s):
    if own:
        import hadamard_rotated_bit_gb300 as h32
        return h32.h32_f8_gemm(s["wq"], s["wd"], s["xq"], s["xd"], y_dtype=DT[s["y"]])
    return (_rows(s) @ _weights(s).t()).to(DT[s["y"]])


def _run_experts(s):
    E, N, K = s["E"], s["N"], s["K"]
    if own:
        import hadamard_rotated_bit_gb300 as h32
        return h32.h32_f8_gemm_experts(s["wq"], s["wd"], s["xq"], s["xd"], s["off"], N,
                                       y_dtype=DT[s["y"]])
    R = s["xq"].shape[0]
    d = s["wd"].reshape(E, -1, s["wd"].shape[1]).repeat_interleave(128, 1)[:, :N]
    w = s["wq"].view(F8).float().reshape(E, N, K) * d.repeat_interleave(128, 2)[:, :, :K]
    r = torch.arange(R, device=w.device)
    e = (r[:, None] >= s["off"][None, 1:]).sum(1)      # the row's expert, and its place there
    at = r - s["off"][e]
    x = torch.zeros((E, s["most"], K), device=w.device)
    x[e, at] = _rows(s)
    return (x @ w.transpose(1, 2))[e, at].to(DT[s["y"]])


def _run_logprobs(s):
    top = s["top"]
    if own:
        import hadamard_rotated_bit_gb300 as h32
        lp, ent, ids, tlp = h32.h32_token_logprobs(s["logits"], s["targets"], top=top)
        return {"logprob": lp, "entropy": ent, "top_id": ids, "top_logprob": tlp}
    l = s["logits"].float()
    m = l.amax(1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)             # (an empty row: every term 0)
    p = torch.exp(l - m)
    S = p.double().sum(1, keepdim=True)
    lse = (m.double() + torch.log(S))                  # -inf for an empty row
    # sum of p log p; a masked token adds 0
    ent = torch.where(S > 0, torch.log(S) - torch.where(p > 0, p * (l - m), 0.0).double().sum(1, keepdim=True) / S,
                      0.0)[:, 0].float()
    order = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :top]

    def at(ids):
        x = l.gather(1, ids)
        return torch.where(x > -math.inf, x.double() - lse, -math.inf).float()

    lp = None
    if s["targets"] is not None:
        t = s["targets"].long()
        lp = torch.where(t >= 0, at(t.clamp_min(0)), 0.0)
    return {"logprob": lp, "entropy": ent, "top_id": order.to(torch.int32), "top_logprob": at(order)}


_RUN = {"quant": _run_quant, "product": _run_product, "experts": _run_experts, "logprobs": _run_logprobs}


# ----------------------------------------------------------------------------
# what a pass cannot do without
# ----------------------------------------------------------------------------
def work(case):
    c = case
    size = {"bf16": 2, "f32": 4}
    if c["op"] == "quant":
        M, K = c["M"], c["K"]
        out = (c["R"] or M) * K
        turn = int(math.log2(c["rotate"])) + 1 if c["rotate"] else 0
        nb = (K + 127) // 128
        d = (out // K if c["kind"] == "act" else (M + 127) // 128) * nb
        read = min(M, c["R"]) * K if c["R"] else M * K
        return {"bytes": read * size[c["x"]] + 4 * c["R"] + out + 4 * d, "flops": out * (2 + turn)}
    if c["op"] == "product":
        M, N, K = c["M"], c["N"], c["K"]
        nb = (K + 127) // 128
        return {"bytes": N * K + M * K + 4 * nb * (M + (N + 127) // 128) + size[c["y"]] * M * N,
                "flops": 2 * M * N * K}
    if c["op"] == "experts":
        R, E, N, K = c["T"] * c["k"], c["E"], c["N"], c["K"]
        # experts that get a row, of E drawn k at a time
        used = E * (1.0 - (1.0 - c["k"] / E) ** c["T"])
        return {"bytes": used * N * K + R * K + 4 * (K + 127) // 128 * R + 4 * (E + 1)
                + size[c["y"]] * R * N, "flops": 2 * R * N * K}
    T, V = c["T"], c["V"]
    return {"bytes": T * (V * size[c["x"]] + 8 * c["n"] + 4 + 8 * c["top"]), "flops": 5 * T * V}


# ----------------------------------------------------------------------------
# the definitions in 64 bits
# ----------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"quant": _exact_quant, "product": _exact_product, "experts": _exact_experts,
            "logprobs": _exact_logprobs}[s["op"]](s)


def _e4m3(q):
    """The e4m3 number nearest to q, ties to the even one, in 64 bits: steps of 2^(e - 3)
    from 2^e on, of 2^-9 below 2^-6; at most 448."""
    e = torch.frexp(q).exponent.clamp_min(-5) - 1
    step = torch.ldexp(torch.ones_like(q), e - 3)
    return (torch.round(q / step) * step).clamp(-448.0, 448.0)


def _exact_quant(s):
    v = s["x_t"]
    if s["rows"] is not None:
        v = torch.index_select(v, 0, s["rows"])
    v = v.to(torch.float64)
    R, K = v.shape
    half = 1
    while half < s["rotate"]:   # the butterfly of the transform, stride by stride
        p = v.reshape(R, -1, 2, half)
        v = torch.stack((p[:, :, 0] + p[:, :, 1], p[:, :, 0] - p[:, :, 1]), 2).reshape(R, K)
        half *= 2
    v = v / math.sqrt(s["rotate"] or 1)
    tall = 1 if s["kind"] == "act" else 128
    codes = torch.empty_like(v)
    scales = torch.empty((-(-R // tall), -(-K // 128)), dtype=torch.float64, device=v.device)
    for b in range(scales.shape[1]):
        part = v[:, 128 * b:128 * b + 128]
        big = part.abs().amax(1)
        big = torch.nn.functional.pad(big, (0, -R % tall)).reshape(-1, tall).amax(1)
        scales[:, b] = big / 448.0
        per = (big / 448.0).repeat_interleave(tall)[:R, None]
        codes[:, 128 * b:128 * b + 128] = _e4m3(part / per.clamp_min(1e-300))
    return {"codes": codes, "scales": scales.t().contiguous() if tall == 1 else scales}


def _exact_blocks(wq, wd, xq, xd):
    """Block by block: (x_codes . w_codes) times the two scales, in 64 bits."""
    y = torch.zeros((xq.shape[0], wq.shape[0]), dtype=torch.float64, device=wq.device)
    for b in range(wd.shape[1]):
        cols = slice(128 * b, 128 * b + 128)
        w = wq[:, cols].view(F8).double()
        w *= wd[:, b].double().repeat_interleave(128)[:w.shape[0], None]
        x = xq[:, cols].view(F8).double()
        x *= xd[b, :x.shape[0], None].double()
        y.addmm_(x, w.t())
    return y


def _exact_product(s):
    return _exact_blocks(s["wq"], s["wd"], s["xq"], s["xd"])


def _exact_experts(s):
    E, N = s["E"], s["N"]
    tall = s["wd"].shape[0] // E
    off = s["off"].tolist()
    parts = [_exact_blocks(s["wq"][e * N:(e + 1) * N], s["wd"][e * tall:(e + 1) * tall],
                           s["xq"][off[e]:off[e + 1]], s["xd"][:, off[e]:off[e + 1]])
             for e in range(E)]
    return torch.cat(parts, 0)


def _exact_logprobs(s):
    T, top = s["T"], s["top"]
    out = {"logprob": [], "entropy": [], "top_id": [], "top_logprob": []}
    for r0 in range(0, T, 256):
        l = s["logits"][r0:r0 + 256].double()
        empty = torch.isinf(l).all(1, keepdim=True)
        lse = torch.logsumexp(torch.where(empty, 0.0, l), 1, keepdim=True)
        lp = torch.where(empty, -math.inf, l - lse)
        pr = torch.exp(lp)
        out["entropy"].append(-torch.special.xlogy(pr, pr).sum(1))
        ids = torch.argsort(lp, dim=1, descending=True, stable=True)[:, :top]
        out["top_id"].append(ids)
        out["top_logprob"].append(torch.take_along_dim(lp, ids, 1))
        if s["targets"] is not None:
            t = s["targets"][r0:r0 + 256].long()
            x = torch.take_along_dim(lp, t.clamp_min(0), 1)
            out["logprob"].append(torch.where(t < 0, 0.0, x))
    done = {k: torch.cat(v, 0) if v else None for k, v in out.items()}
    done["top_id"] = done["top_id"].to(torch.int32)
    return done
