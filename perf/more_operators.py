"""The operators of a feed-forward block of quantised layers, dense or of many
experts: what is measured, their plain forms and their definitions in 64 bits.

  act       out = act(x W^T + bias) (+ residual), or gated: the rows of W are
            [gate; up] and out = act(x W_gate^T) * (x W_up^T); where the block is
            trained, z = x W^T + bias is kept too
  act_bwd   dz and the bias's gradient from dy and a kept z
  route     one training pass of a router and the sum that it weights: ids and
            weights from the logits, out = residual + sum_j w_j y_j, then dy and
            the logits' gradient from dout
  moe       a block of experts in serving: route, gated product, product back,
            weighted sum
  experts   one training pass of the experts' products: y with z kept, then the
            gradient of the block's input from dy

Widths are those of the layers in this repository's workloads (512, 4096, 14336)
and generic ones.  Stacked experts are one layer of E * N rows.
"""
import math

import torch

own = False             # True: the framework's operators; False: their plain forms

CODE_BITS = {"any4": 4, "int4": 4, "any2": 2, "any3": 3}
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def _act(fmt, M, N, K, g, act, gate=False, bias=False, residual=False, keep=False):
    return {"op": "act", "fmt": fmt, "M": M, "N": N, "K": K, "g": g, "act": act, "gate": gate, "bias": bias,
            "residual": residual, "keep": keep}


def listed():
    return [
        # one token's gate and up projections: weights streamed, latency
        {"name": "act_decode_1", **_act("any4", 1, 28672, 4096, 128, "silu", gate=True)},
        # sixteen requests' down projection onto the residual stream, 2-bit codes
        {"name": "act_decode_16", **_act("any2", 16, 4096, 14336, 1024, "none", bias=True, residual=True)},
        # the forward pass of a training step through gate and up, z kept
        {"name": "act_keep_4096", **_act("any4", 4096, 28672, 4096, 128, "silu", gate=True, keep=True)},
        # the smallest training batch of the workloads, and the long one
        {"name": "act_bwd_64", "op": "act_bwd", "M": 64, "N": 512, "act": "gelu", "gate": False, "bias": True},
        {"name": "act_bwd_4096", "op": "act_bwd", "M": 4096, "N": 28672, "act": "silu", "gate": True, "bias": True},
        # an odd short batch over few experts, bf16 logits; a long one over many in groups
        {"name": "route_33", "op": "route", "T": 33, "E": 8, "k": 2, "D": 512, "score": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "renorm": True, "bf16": True},
        {"name": "route_8192", "op": "route", "T": 8192, "E": 256, "k": 8, "D": 2048, "score": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "renorm": True, "bf16": False},
        # one token through two of eight wide experts; a decode batch over many narrow
        # ones; prompts, an odd number of tokens
        {"name": "moe_decode_1", "op": "moe", "fmt": "any4", "T": 1, "E": 8, "k": 2, "D": 4096, "F": 14336, "g": 128},
        {"name": "moe_decode_32", "op": "moe", "fmt": "any4", "T": 32, "E": 64, "k": 8, "D": 2048, "F": 1024, "g": 128},
        {"name": "moe_prefill_1031", "op": "moe", "fmt": "any4", "T": 1031, "E": 8, "k": 2, "D": 4096, "F": 14336,
         "g": 128},
        # training through frozen experts: an odd small batch of plain int4 and a long one
        {"name": "experts_37", "op": "experts", "fmt": "int4", "T": 37, "E": 4, "k": 2, "D": 512, "F": 512, "g": 128},
        {"name": "experts_2048", "op": "experts", "fmt": "any4", "T": 2048, "E": 16, "k": 4, "D": 2048, "F": 1024,
         "g": 256},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["act", "act", "act_bwd", "route", "moe", "moe", "experts"])
    if op in ("act", "act_bwd"):
        M, gate = _log(rng, 1, 4096), rng.random() < 0.5
        N = 2 * _log(rng, 8, 14336) if gate else _log(rng, 16, 14336)
        act, bias = rng.choice(ACTS[1:]), rng.random() < 0.5
        if op == "act_bwd":
            return {"op": op, "M": M, "N": N, "act": act, "gate": gate, "bias": bias}
        K = 128 * _log(rng, 1, 32 if gate else 112)
        g = 128 * rng.choice([d for d in range(1, 9) if (K // 128) % d == 0])
        M = min(M, int(4.8e11 // (N * K)))
        return _act(rng.choice(sorted(CODE_BITS)), M, N, K, g, act, gate, bias, rng.random() < 0.5, rng.random() < 0.5)
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, 2, 256 // groups)
        top = rng.randint(1, groups)
        k = rng.randint(1, min(8, top * E // groups))
        score = rng.choice(["softmax", "sigmoid"])
        return {"op": op, "T": _log(rng, 1, 8192), "E": E, "k": k, "D": 8 * _log(rng, 16, 256), "score": score,
                "bias": rng.random() < 0.5, "groups": groups, "top_groups": top,
                "renorm": k > 1 and rng.random() < 0.7, "bf16": rng.random() < 0.5}
    E = _log(rng, 2, 64)
    k = rng.randint(1, min(8, E))
    D, F = 128 * _log(rng, 1, 32), 128 * _log(rng, 1, max(1, min(112, 512 // E)))
    g = 128 * rng.choice([d for d in (1, 2, 4) if (D // 128) % d == 0 and (F // 128) % d == 0])
    T = max(1, min(_log(rng, 1, 2048), int(1.2e12 // (E * D * F * (2 + (k if op == "moe" else 4 * k))))))
    return {"op": op, "fmt": rng.choice(sorted(CODE_BITS)), "T": T, "E": E, "k": k, "D": D, "F": F, "g": g}


def _layer_bytes(fmt, N, K, g):
    return N * K * CODE_BITS[fmt] // 8 + 4 * N * (K // g) + (0 if fmt == "int4" else 32 * N)


def work(case):
    op = case["op"]
    if op in ("act", "act_bwd"):
        M, N = case["M"], case["N"]
        No = N // 2 if case["gate"] else N
        if op == "act_bwd":     # dy and z in, dz and the bias's gradient out
            return {"bytes": 2 * M * (No + 2 * N) + (4 * N if case["bias"] else 0), "flops": 10 * M * N}
        K = case["K"]
        rows = K + No * (2 if case["residual"] else 1) + (N if case["keep"] else 0)
        return {"bytes": _layer_bytes(case["fmt"], N, K, case["g"]) + 2 * M * rows + (2 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    T, E, k, D = case["T"], case["E"], case["k"], case["D"]
    if op == "route":           # logits, y (twice), residual, dout in; w, ids, out, dy, dlogits out
        return {"bytes": (2 if case["bf16"] else 4) * 2 * T * E + 12 * T * k + 2 * T * D * (3 * k + 3),
                "flops": 6 * T * k * D + 20 * T * E}
    F, g, fmt = case["F"], case["g"], case["fmt"]
    used = E * (1 - (1 - k / E) ** T)
    layers = used * (_layer_bytes(fmt, 2 * F, D, g) + _layer_bytes(fmt, D, F, g))
    if op == "moe":             # x and logits in, the block's output out
        return {"bytes": layers + 4 * T * D + 4 * T * E, "flops": 6 * T * k * D * F}
    # forward and backward: x, dy, ids in; z kept and read, y and dx out
    return {"bytes": 2 * layers + 2 * T * D * (2 + 2 * k) + 8 * T * k * F + 4 * T * k, "flops": 12 * T * k * D * F}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def _activation(g, M, K):
    """Rows of a normal distribution with one channel in a hundred 20 times larger."""
    x = _normal(g, M, K)
    big = torch.randperm(K, generator=g, device="cuda")[: round(0.01 * K)]
    x[:, big] *= 20
    return x.to(torch.bfloat16)


def _layer(g, fmt, N, K, group):
    """A layer with outputs of about the size of 1 for inputs of _activation
    or of the size of 1."""
    bits = CODE_BITS[fmt]
    code = torch.randint(0, 1 << bits, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    alpha = (0.5 + torch.rand(N, K // group, generator=g, device="cuda")) * K ** -0.5
    if fmt == "int4":           # codes 0 .. 15 about their mean
        beta = -7.5 * alpha
        alpha = alpha * 0.2
        beta = beta * 0.2
    else:
        beta = _normal(g, N, K // group, std=0.1 * K ** -0.5)
    return {"packed": _pack(code, bits), "lut": _normal(g, N, 16).sort(dim=1).values.to(torch.bfloat16),
            "alpha": alpha.to(torch.bfloat16), "beta": beta.to(torch.bfloat16)}


def _logits(g, case):
    """A router's logits: some experts are more popular than others."""
    l = _normal(g, case["T"], case["E"], std=1.5) + _normal(g, case["E"], std=0.5)
    return l.to(torch.bfloat16) if case.get("bf16") else l


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed))
    s = {"case": dict(case)}
    op = case["op"]
    if op in ("act", "act_bwd"):
        M, N = case["M"], case["N"]
        No = N // 2 if case["gate"] else N
        if op == "act_bwd":
            s["z"] = _normal(g, M, N, std=1.5).to(torch.bfloat16)
            s["dy"] = _normal(g, M, No, std=0.01).to(torch.bfloat16)
            return s
        s["x"] = _activation(g, M, case["K"])
        s["layer"] = _layer(g, case["fmt"], N, case["K"], case["g"])
        s["bias"] = _normal(g, N, std=0.2).to(torch.bfloat16) if case["bias"] else None
        s["residual"] = _normal(g, M, No, std=2.0).to(torch.bfloat16) if case["residual"] else None
        return s
    T, E, k, D = case["T"], case["E"], case["k"], case["D"]
    if op == "route":
        s["logits"] = _logits(g, case)
        s["bias"] = _normal(g, E, std=0.05) if case["bias"] else None
        s["y"] = _normal(g, T, k, D).to(torch.bfloat16)
        s["residual"] = _normal(g, T, D, std=2.0).to(torch.bfloat16)
        s["dout"] = _normal(g, T, D, std=0.01).to(torch.bfloat16)
        return s
    F = case["F"]
    s["x"] = _activation(g, T, D)
    s["up"] = _stack(_layer(g, case["fmt"], E * 2 * F, D, case["g"]), E)
    s["down"] = _stack(_layer(g, case["fmt"], E * D, F, case["g"]), E)
    s["logits"] = _logits(g, case)
    if op == "experts":
        s["ids"] = torch.sort(s["logits"], dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32).contiguous()
        s["dy"] = _normal(g, T, k, D, std=0.01).to(torch.bfloat16)
    return s


def _stack(layer, E):
    return {"packed": layer["packed"], **{n: layer[n].view(E, -1, layer[n].shape[1]) for n in ("lut", "alpha", "beta")}}


def _pack(code, bits):
    """Codes [N, K] in the packed layout of a layer: tiles of 16 rows x 128 k,
    in each of which the 64 slots of 32 codes follow one another."""
    N, K = code.shape
    rows = -(-N // 16) * 16
    code = torch.cat([code, code.new_zeros(rows - N, K)]) if rows > N else code
    slots = code.view(rows // 16, 16, K // 128, 4, 32).permute(0, 2, 3, 1, 4)
    if bits == 4:
        out = slots[..., 0::2] | slots[..., 1::2] << 4
    elif bits == 2:
        out = slots[..., 0::4] | slots[..., 1::4] << 2 | slots[..., 2::4] << 4 | slots[..., 3::4] << 6
    else:
        pair = slots[..., 0::2] | slots[..., 1::2] << 3
        j = torch.arange(12, device=code.device)
        top = pair[..., 12 + j % 4] >> (2 * (j // 4)).to(torch.uint8) & 3
        out = pair[..., :12] | top << 6
    return out.contiguous().view(-1)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    case = s["case"]
    return {"act": _run_act, "act_bwd": _run_act_bwd, "route": _run_route, "moe": _run_moe,
            "experts": _run_experts}[case["op"]](s, case)


def _tables(fmt, layer):
    return (layer["packed"],) + (() if fmt == "int4" else (layer["lut"],)) + (layer["alpha"], layer["beta"])


def _unpack(packed, N, K, bits):
    """The codes [N, K] of a packed layer."""
    b = packed.view(-(-N // 16), K // 128, 4, 16, bits * 4)
    if bits == 4:
        code = torch.stack([b & 15, b >> 4], dim=-1)
    elif bits == 2:
        code = torch.stack([b & 3, b >> 2 & 3, b >> 4 & 3, b >> 6], dim=-1)
    else:
        top = (b >> 6).view(*b.shape[:-1], 3, 4)
        pair = torch.cat([b & 63, top[..., 0, :] | top[..., 1, :] << 2 | top[..., 2, :] << 4], dim=-1)
        code = torch.stack([pair & 7, pair >> 3], dim=-1)
    return code.reshape(*b.shape[:-1], 32).permute(0, 3, 1, 2, 4).reshape(-1, K)[:N]


def _weights(layer, fmt, g):
    """W [N, K] in 32 bits; stacked experts one after another."""
    lut, alpha, beta = (layer[n].reshape(-1, layer[n].shape[-1]) for n in ("lut", "alpha", "beta"))
    N, K = alpha.shape[0], alpha.shape[1] * g
    code = _unpack(layer["packed"], N, K, CODE_BITS[fmt])
    v = code.float() if fmt == "int4" else torch.gather(lut.float(), 1, code.long())
    v = v.view(N, -1, g) * alpha.float()[:, :, None] + beta.float()[:, :, None]
    return v.to(torch.bfloat16).float().view(N, K)       # a weight is a bf16 value


def _f(act, z):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))


def _slope(act, z):
    if act == "none":
        return torch.ones_like(z)
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    c = 2 * math.sqrt(2 / math.pi)
    p = 1 / (1 + torch.exp(-c * (z + 0.044715 * z ** 3)))
    return p + z * p * (1 - p) * c * (1 + 3 * 0.044715 * z * z)


def _activate(z, act, gate):
    if not gate:
        return _f(act, z)
    F = z.shape[-1] // 2
    return _f(act, z[..., :F]) * z[..., F:]


def _activate_bwd(dy, z, act, gate):
    if not gate:
        return dy * _slope(act, z)
    F = z.shape[-1] // 2
    return torch.cat([dy * z[..., F:] * _slope(act, z[..., :F]), dy * _f(act, z[..., :F])], dim=-1)


def _run_act(s, case):
    fmt, g, act, gate = case["fmt"], case["g"], case["act"], case["gate"]
    if own:
        import gemm_any4_amd as any4

        call = {"any4": any4.gemm_act, "int4": any4.gemm_int4_act, "any2": any4.any2_gemm_act,
                "any3": any4.any3_gemm_act}[fmt]
        z = torch.empty((case["M"], case["N"]), dtype=torch.bfloat16, device=s["x"].device) if case["keep"] else None
        y = call(s["x"], *_tables(fmt, s["layer"]), g, act=act, gate=gate, bias=s["bias"], residual=s["residual"], z=z)
        return {"y": y, "z": z}
    z = s["x"].float() @ _weights(s["layer"], fmt, g).t()
    if case["bias"]:
        z = z + s["bias"].float()
    y = _activate(z, act, gate)
    if case["residual"]:
        y = y + s["residual"].float()
    return {"y": y.to(torch.bfloat16), "z": z.to(torch.bfloat16) if case["keep"] else None}


def _run_act_bwd(s, case):
    if own:
        import gemm_any4_amd as any4

        dz, dbias = any4.act_backward(s["dy"], s["z"], act=case["act"], gate=case["gate"], need_bias=case["bias"])
        return {"dz": dz, "dbias": dbias}
    dz = _activate_bwd(s["dy"].float(), s["z"].float(), case["act"], case["gate"])
    return {"dz": dz.to(torch.bfloat16), "dbias": dz.double().sum(dim=0).float() if case["bias"] else None}


def _scores(l, kind):
    if kind == "sigmoid":
        return 1 / (1 + torch.exp(-l))
    e = torch.exp(l - l.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _choose(l, bias, kind, k, groups, top_groups):
    """(scores, the k experts) in 64 bits, since a bit decides between two experts."""
    l = l.double()
    p = _scores(l, kind)
    choice = p if bias is None else p + bias.double()
    rank = l if bias is None else choice        # the same order, without a score's rounding
    if top_groups < groups:
        T, E = l.shape
        best = choice.view(T, groups, -1).sort(dim=2, descending=True).values[:, :, :2].sum(dim=2)
        order = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :top_groups]
        kept = torch.zeros(T, groups, dtype=torch.bool, device=l.device).scatter(1, order, True)
        rank = torch.where(kept.repeat_interleave(E // groups, dim=1), rank, torch.full_like(rank, -math.inf))
    return p, torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :k]


def _route(s, case):
    """(weights, ids, scores) in 64 bits."""
    p, ids = _choose(s["logits"], s.get("bias"), case.get("score", "softmax"), case["k"], case.get("groups", 1),
                     case.get("top_groups", 1))
    w = p.gather(1, ids)
    return w / w.sum(dim=1, keepdim=True) if case.get("renorm", True) else w, ids, p


def _route_bwd(dw, w, ids, p, case):
    """The logits' gradient from that of the weights."""
    chosen = p.gather(1, ids)
    ds = dw
    if case["renorm"]:
        ds = (dw - (dw * w).sum(dim=1, keepdim=True)) / chosen.sum(dim=1, keepdim=True)
    ds = torch.zeros_like(p).scatter(1, ids, ds)
    if case["score"] == "sigmoid":
        return ds * p * (1 - p)
    return p * (ds - (ds * p).sum(dim=1, keepdim=True))


def _run_route(s, case):
    if own:
        import gemm_any4_amd as any4

        how = {"score": case["score"], "renorm": case["renorm"]}
        w, ids = any4.route(s["logits"], case["k"], bias=s["bias"], groups=case["groups"],
                            top_groups=case["top_groups"], **how)
        out = any4.combine(s["y"], w, residual=s["residual"])
        dy, dw = any4.combine_backward(s["dout"], s["y"], w)
        return {"w": w, "ids": ids, "out": out, "dy": dy, "dlogits": any4.route_backward(dw, s["logits"], ids, **how)}
    w, ids, p = _route(s, case)
    y, dout, w32 = s["y"].float(), s["dout"].float(), w.float()
    out = s["residual"].float() + (w32[:, :, None] * y).sum(dim=1)
    dw = (dout[:, None, :] * y).sum(dim=2)
    dlogits = _route_bwd(dw.double(), w, ids, p, case)
    return {"w": w32, "ids": ids.to(torch.int32), "out": out.to(torch.bfloat16),
            "dy": (w32[:, :, None] * dout[:, None, :]).to(torch.bfloat16), "dlogits": dlogits.to(s["logits"].dtype)}


def _through(x, W, ids, E):
    """x [T, k or 1, K] through the experts [E * N, K] that ids [T, k] names: every
    row through every expert, of which its own is taken."""
    T, k = ids.shape
    z = (x.reshape(-1, x.shape[2]) @ W.t()).view(T, x.shape[1], E, -1)
    return torch.gather(z.expand(T, k, *z.shape[2:]), 2, ids.long()[:, :, None, None].expand(T, k, 1, z.shape[3]))[:, :, 0]


def _back(dz, W, ids, E):
    """dz [T, k, N] back through the experts [E * N, K]."""
    W = W.view(E, -1, W.shape[1]).transpose(1, 2).reshape(-1, W.shape[0] // E)
    return _through(dz, W, ids, E)


def _experts_call(fmt):
    import gemm_any4_amd as any4

    return {"any4": any4.experts_gemm, "int4": any4.experts_gemm_int4, "any2": any4.any2_experts_gemm,
            "any3": any4.any3_experts_gemm}[fmt]


def _between(case, n, device):
    """For n columns of what lies between two products, in two bf16 parts: rows of a product need not
    be rounded to bf16, whatever the number of pairs."""
    return torch.empty((2, case["T"], case["k"], n), dtype=torch.bfloat16, device=device)


def _run_moe(s, case):
    fmt, g, E = case["fmt"], case["g"], case["E"]
    if own:
        import gemm_any4_amd as any4

        call = _experts_call(fmt)
        w, ids = any4.route(s["logits"], case["k"])
        plan = any4.experts_plan(ids, E)
        h = _between(case, case["F"], ids.device)
        call(s["x"], *_tables(fmt, s["up"]), g, ids, act="silu", gate=True, plan=plan, out=h)
        y = torch.empty((case["T"], case["k"], case["D"]), dtype=torch.float32, device=ids.device)
        return any4.combine(call(h, *_tables(fmt, s["down"]), g, ids, plan=plan, out=y), w)
    w, ids, _ = _route(s, case)
    h = _activate(_through(s["x"].float()[:, None], _weights(s["up"], fmt, g), ids, E), "silu", True)
    y = _through(h, _weights(s["down"], fmt, g), ids, E)
    return (w.float()[:, :, None] * y).sum(dim=1).to(torch.bfloat16)


def _run_experts(s, case):
    fmt, g, E, T, k = case["fmt"], case["g"], case["E"], case["T"], case["k"]
    ids = s["ids"]
    if own:
        import gemm_any4_amd as any4

        call = _experts_call(fmt)
        back = {"any4": any4.experts_gemm_dx, "int4": any4.experts_gemm_int4_dx, "any2": any4.any2_experts_gemm_dx,
                "any3": any4.any3_experts_gemm_dx}[fmt]
        plan = any4.experts_plan(ids, E)
        # z and the rows' gradients are kept in fp32, what enters a product in parts
        z, dh, dx = (torch.empty((T, k, n), dtype=torch.float32, device=ids.device)
                     for n in (2 * case["F"], case["F"], case["D"]))
        h, dz = (_between(case, n, ids.device) for n in (case["F"], 2 * case["F"]))
        call(s["x"], *_tables(fmt, s["up"]), g, ids, act="silu", gate=True, z=z, plan=plan, out=h)
        y = call(h, *_tables(fmt, s["down"]), g, ids, plan=plan)
        back(s["dy"], *_tables(fmt, s["down"]), g, ids, plan=plan, out=dh)
        any4.act_backward(dh, z, act="silu", gate=True, need_bias=False, dz=dz)
        back(dz, *_tables(fmt, s["up"]), g, ids, plan=plan, out=dx)
        return {"y": y, "dx": any4.combine(dx)}
    up, down = _weights(s["up"], fmt, g), _weights(s["down"], fmt, g)
    z = _through(s["x"].float()[:, None], up, ids, E)
    y = _through(_activate(z, "silu", True), down, ids, E)
    dh = _back(s["dy"].float(), down, ids, E)
    dx = _back(_activate_bwd(dh, z, "silu", True), up, ids, E).sum(dim=1)
    return {"y": y.to(torch.bfloat16), "dx": dx.to(torch.bfloat16)}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"act": _exact_act, "act_bwd": _exact_act_bwd, "route": _exact_route, "moe": _exact_moe,
            "experts": _exact_experts}[case["op"]](s, case)


def _exact_weights(layer, fmt, g, e=None):
    """W [N, K] of a layer or of expert e: alpha * value + beta in 64 bits (exact but
    for far exponents), rounded to 32 bits and then to the bf16 that a weight is."""
    lut, alpha, beta = ((layer[n] if e is None else layer[n][e]).double() for n in ("lut", "alpha", "beta"))
    bits, (N, K) = CODE_BITS[fmt], (alpha.shape[0], alpha.shape[1] * g)
    n = torch.arange(N, device="cuda")[:, None] + (0 if e is None else e * N)
    k = torch.arange(K, device="cuda")[None, :]
    # slot of 32 codes: row block, chunk of 128 k, quarter of it, row in the block
    slot = ((n // 16 * (K // 128) + k // 128) * 4 + k % 128 // 32) * 16 + n % 16
    i, size, packed = k % 32, 4 * bits, layer["packed"]
    if bits == 3:
        p = i // 2
        low = packed[slot * size + p.clamp(max=11)].long() & 63
        j = (p - 12).clamp(min=0)
        t = [packed[slot * size + j + 4 * q].long() >> 6 << 2 * q for q in range(3)]
        code = torch.where(p < 12, low, t[0] + t[1] + t[2]) >> 3 * (i % 2) & 7
    else:
        per = 8 // bits
        code = packed[slot * size + i // per].long() >> bits * (i % per) & (1 << bits) - 1
    value = code.double() if fmt == "int4" else lut.gather(1, code)
    w = alpha.repeat_interleave(g, 1) * value + beta.repeat_interleave(g, 1)
    return w.float().to(torch.bfloat16).double()


def _exact_f(act, z):
    """(act(z), act'(z)) from the functions' definitions."""
    one = torch.ones_like(z)
    if act == "none":
        return z, one
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "silu":
        p = torch.special.expit(z)
        return z * p, p + z * p * (1 - p)
    if act == "gelu":
        p = torch.special.ndtr(z)
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    c, d = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(c * (z + d * z ** 3))
    return z * (1 + t) / 2, (1 + t) / 2 + z / 2 * (1 - t * t) * c * (1 + 3 * d * z * z)


def _exact_activate(z, act, gate):
    if not gate:
        return _exact_f(act, z)[0]
    a, b = z.chunk(2, dim=-1)
    return _exact_f(act, a)[0] * b


def _exact_dz(dy, z, act, gate):
    if not gate:
        return dy * _exact_f(act, z)[1]
    a, b = z.chunk(2, dim=-1)
    v, slope = _exact_f(act, a)
    return torch.cat([dy * b * slope, dy * v], dim=-1)


def _exact_act(s, case):
    z = s["x"].double() @ _exact_weights(s["layer"], case["fmt"], case["g"]).t()
    if case["bias"]:
        z += s["bias"].double()
    y = _exact_activate(z, case["act"], case["gate"])
    return {"y": y + s["residual"].double() if case["residual"] else y, "z": z if case["keep"] else None}


def _exact_act_bwd(s, case):
    dz = _exact_dz(s["dy"].double(), s["z"].double(), case["act"], case["gate"])
    return {"dz": dz, "dbias": dz.sum(dim=0) if case["bias"] else None}


def _exact_choice(s, case):
    """(weights, ids, scores): experts taken one after another."""
    l = s["logits"].double()
    T, E = l.shape
    p = torch.special.expit(l) if case.get("score") == "sigmoid" else torch.softmax(l, dim=1)
    bias = s.get("bias")
    choice = p if bias is None else p + bias.double()
    left = (l if bias is None else choice).clone()
    groups, top = case.get("groups", 1), case.get("top_groups", 1)
    if top < groups:
        best = torch.topk(choice.view(T, groups, -1), min(2, E // groups), dim=2).values.sum(dim=2)
        out = torch.ones(T, groups, dtype=torch.bool, device=l.device)
        for _ in range(top):
            i = best.argmax(dim=1, keepdim=True)
            out.scatter_(1, i, False)
            best.scatter_(1, i, -math.inf)
        left.view(T, groups, -1)[out] = -math.inf
    ids = []
    for _ in range(case["k"]):
        highest = left == left.amax(dim=1, keepdim=True)
        ids.append(torch.where(highest, torch.arange(E, device=l.device), E).amin(dim=1, keepdim=True))
        left.scatter_(1, ids[-1], -math.inf)
    ids = torch.cat(ids, dim=1)
    w = p.gather(1, ids)
    return w / w.sum(dim=1, keepdim=True) if case.get("renorm", True) else w, ids, p


def _exact_route(s, case):
    w, ids, p = _exact_choice(s, case)
    y, dout = s["y"].double(), s["dout"].double()
    out = s["residual"].double() + torch.bmm(w[:, None], y)[:, 0]
    dw = torch.bmm(y, dout[:, :, None])[:, :, 0]
    T, E, k = case["T"], case["E"], case["k"]
    # d w_i / d s_j, then d s_j / d l_e
    pick = torch.zeros(T, k, E, dtype=torch.float64, device=y.device).scatter_(2, ids[:, :, None], 1.0)
    chosen = p.gather(1, ids)
    ds = dw
    if case["renorm"]:
        total = chosen.sum(dim=1, keepdim=True)
        ds = dw / total - torch.bmm(dw[:, None], chosen[:, :, None])[:, :, 0] / total ** 2
    ds = torch.bmm(ds[:, None], pick)[:, 0]
    if case["score"] == "sigmoid":
        dl = ds * torch.exp(-torch.log1p(torch.exp(-s["logits"].double())) - torch.log1p(torch.exp(s["logits"].double())))
    else:
        dl = ds * p - p * torch.bmm(ds[:, None], p[:, :, None])[:, :, 0]
    return {"w": w, "ids": None, "out": out, "dy": w[:, :, None] * dout[:, None, :], "dlogits": dl}


def _exact_rows(s, case, ids, x, dy=None):
    """Pair by pair, one expert at a time: y, and dx of the pairs."""
    fmt, g, k = case["fmt"], case["g"], case["k"]
    flat = ids.reshape(-1)
    y = torch.zeros(flat.numel(), case["D"], dtype=torch.float64, device=x.device)
    dx = torch.zeros_like(y)
    for e in torch.unique(flat).tolist():
        rows = torch.nonzero(flat == e).flatten()
        up, down = _exact_weights(s["up"], fmt, g, e), _exact_weights(s["down"], fmt, g, e)
        z = x[rows // k] @ up.t()
        y[rows] = _exact_activate(z, "silu", True) @ down.t()
        if dy is not None:
            dx[rows] = _exact_dz(dy[rows] @ down, z, "silu", True) @ up
    return y, dx


def _exact_moe(s, case):
    w, ids, _ = _exact_choice(s, case)
    y, _ = _exact_rows(s, case, ids, s["x"].double())
    return torch.bmm(w[:, None], y.view(*ids.shape, -1))[:, 0]


def _exact_experts(s, case):
    T, k, D = case["T"], case["k"], case["D"]
    y, dx = _exact_rows(s, case, s["ids"], s["x"].double(), s["dy"].double().view(T * k, D))
    return {"y": y.view(T, k, D), "dx": dx.view(T, k, D).sum(dim=1)}
