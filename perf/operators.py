"""The operators around a frozen any4 layer that is served with, or trained
through, low-rank adapters: what is measured, their plain forms and their
definitions in 64 bits.

  lora      y' = y + s_a (x A_a^T) B_a, every row with the adapter of its request
  train     one training pass of the adapters: the forward that keeps h = x A_a^T
            (and x, or x in 8 bits), then dx, dA and dB from dy
  act8      an activation kept in 8 bits (one scale per 128 channels) and read back
  gemm_dx   dx = dy W, the gradient of a quantised layer's input

Sizes are those of the layers in this repository's workloads (512x512,
4096x4096, 14336x4096, 4096x14336) and generic ones.  A is [L, r, K] and B is
[L, r, N]: L adapters of rank r.
"""
import math

import torch

own = False             # True: the framework's operators; False: their plain forms

GROUP = 128             # channels that share one scale of an 8-bit activation
CODE_BITS = {"any4": 4, "int4": 4, "any2": 2, "any3": 3}


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one request in decode: latency is all there is
        {"name": "lora_decode_1", "op": "lora", "M": 1, "K": 4096, "N": 4096, "r": 16, "L": 8, "ids": "distinct"},
        # sixteen requests, each with a fine-tune of its own
        {"name": "lora_decode_16", "op": "lora", "M": 16, "K": 4096, "N": 14336, "r": 16, "L": 32, "ids": "distinct"},
        # a larger decode batch over a few popular fine-tunes, in no order
        {"name": "lora_decode_48", "op": "lora", "M": 48, "K": 14336, "N": 4096, "r": 64, "L": 8, "ids": "mixed"},
        # prompts of five requests behind one another, an odd number of tokens
        {"name": "lora_prefill_1031", "op": "lora", "M": 1031, "K": 4096, "N": 14336, "r": 32, "L": 5, "ids": "runs"},
        # the smallest training step that the workloads have
        {"name": "train_64", "op": "train", "M": 64, "K": 512, "N": 512, "r": 8, "L": 1, "ids": "runs", "act8": False},
        # a training step of one adapter on the up projection, input kept in 8 bits
        {"name": "train_4096_act8", "op": "train", "M": 4096, "K": 4096, "N": 14336, "r": 16, "L": 1, "ids": "runs",
         "act8": True},
        # four adapters trained at once on a layer with an odd number of outputs
        {"name": "train_2048_four", "op": "train", "M": 2048, "K": 4096, "N": 4099, "r": 64, "L": 4, "ids": "runs",
         "act8": False},
        # a decode batch's activation, and a long batch's wide one
        {"name": "act8_16", "op": "act8", "M": 16, "K": 4096},
        {"name": "act8_8192", "op": "act8", "M": 8192, "K": 14336},
        # the input's gradient: a short batch, a training batch on the up
        # projection, an odd batch through 2-bit codes of the down projection
        {"name": "dx_64", "op": "dx", "fmt": "any4", "M": 64, "N": 4096, "K": 4096, "g": 128},
        {"name": "dx_4096", "op": "dx", "fmt": "any4", "M": 4096, "N": 14336, "K": 4096, "g": 128},
        {"name": "dx_1000_any2", "op": "dx", "fmt": "any2", "M": 1000, "N": 4096, "K": 14336, "g": 1024},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["lora", "lora", "train", "train", "act8", "dx"])
    K = 128 * _log(rng, 1, 112)
    if op == "act8":
        return {"op": op, "M": _log(rng, 1, 8192), "K": K}
    M, N = _log(rng, 1, 4096), _log(rng, 16, 14336)
    if op == "dx":
        g = 128 * rng.choice([d for d in range(1, 9) if (K // 128) % d == 0])
        return {"op": op, "fmt": rng.choice(sorted(CODE_BITS)), "M": M, "N": N, "K": K, "g": g}
    r, L = _log(rng, 1, 128), _log(rng, 1, 64)
    L = max(1, min(L, 2048 // r, int(1e11 // (M * r * (K + N)))))
    ids = rng.choice(["runs", "mixed"] + (["distinct"] if M <= L else []))
    case = {"op": op, "M": M, "K": K, "N": N, "r": r, "L": L, "ids": ids}
    if op == "train":
        case["act8"] = rng.random() < 0.5
    return case


def work(case):
    M, K = case["M"], case["K"]
    if case["op"] == "act8":    # x in, 8 bits and scales out; those in, x out
        return {"bytes": 2 * (2 * M * K + M * K + 4 * M * K // GROUP), "flops": 4 * M * K}
    N = case["N"]
    if case["op"] == "dx":
        layer = N * K * CODE_BITS[case["fmt"]] // 8 + 4 * N * (K // case["g"]) + 32 * N
        return {"bytes": layer + 2 * M * N + 2 * M * K, "flops": 2 * M * N * K}
    r, L = case["r"], case["L"]
    used = min(M, L) if case["ids"] != "mixed" else L * (1 - (1 - 1 / L) ** M)
    adapters = 2 * used * r * (K + N)
    forward = 2 * M * K + 4 * M * N + adapters + 4 * M
    if case["op"] == "lora":
        return {"bytes": forward, "flops": 2 * M * r * (K + N)}
    kept = 4 * M * r + (M * K + 4 * M * K // GROUP if case["act8"] else 0)
    saved = kept + (0 if case["act8"] else 2 * M * K)
    backward = 2 * M * N + saved + 4 * M * K + adapters + 4 * L * r * (K + N)
    return {"bytes": forward + kept + backward, "flops": 6 * M * r * (K + N)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device="cuda") * std


def _activation(g, M, K):
    """Rows of a normal distribution with one channel in a hundred 20 times larger."""
    x = _normal(g, M, K)
    big = torch.randperm(K, generator=g, device="cuda")[: round(0.01 * K)]
    x[:, big] *= 20
    return x.to(torch.bfloat16)


def _ids(g, kind, M, L):
    """The adapter of each row.  "runs": rows of one request behind one another
    (cut at random places); "mixed": any row any adapter; "distinct": another
    adapter for every row.  In larger batches without training, one row in
    sixteen has none (-1)."""
    if kind == "distinct":
        ids = torch.randperm(L, generator=g, device="cuda")[:M]
    elif kind == "mixed":
        ids = torch.randint(0, L, (M,), generator=g, device="cuda")
    else:
        cuts = torch.randint(0, M + 1, (L - 1,), generator=g, device="cuda").sort().values
        ids = torch.searchsorted(cuts, torch.arange(M, device="cuda"), right=True)
    return ids.to(torch.int32)


def prepare(case, seed):
    g = _gen(seed)
    M, K = case["M"], case["K"]
    s = {"case": dict(case)}
    if case["op"] == "act8":
        s["x"] = _activation(g, M, K)
        return s
    N = case["N"]
    if case["op"] == "dx":
        groups = K // case["g"]
        s["dy"] = _normal(g, M, N, std=0.01).to(torch.bfloat16)
        bits = CODE_BITS[case["fmt"]]
        code = torch.randint(0, 1 << bits, (N, K), generator=g, device="cuda", dtype=torch.uint8)
        s["packed"] = _pack(code, bits)
        s["lut"] = _normal(g, N, 16).sort(dim=1).values.to(torch.bfloat16)
        s["alpha"] = (0.005 + 0.015 * torch.rand(N, groups, generator=g, device="cuda")).to(torch.bfloat16)
        s["beta"] = _normal(g, N, groups, std=0.002).to(torch.bfloat16)
        return s
    r, L = case["r"], case["L"]
    s["x"] = _activation(g, M, K)
    s["A"] = _normal(g, L, r, K, std=K ** -0.5).to(torch.bfloat16)
    s["B"] = _normal(g, L, r, N, std=0.05).to(torch.bfloat16)
    s["scale"] = 0.5 + torch.rand(L, generator=g, device="cuda")
    s["ids"] = _ids(g, case["ids"], M, L)
    s["y"] = _normal(g, M, N).to(torch.bfloat16)
    if case["op"] == "lora":
        if M >= 16:
            s["ids"][torch.rand(M, generator=g, device="cuda") < 1 / 16] = -1
        return s
    s["dy"] = _normal(g, M, N, std=0.01).to(torch.bfloat16)
    s["dx"] = _normal(g, M, K, std=0.01).to(torch.bfloat16)
    return s


def _pack(code, bits):
    """Codes [N, K] in the packed layout of a layer: tiles of 16 rows x 128 k,
    in each of which the 64 slots of 32 codes follow one another."""
    N, K = code.shape
    rows = -(-N // 16) * 16
    code = torch.cat([code, code.new_zeros(rows - N, K)])
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
    return {"lora": _lora, "train": _train, "act8": _act8, "dx": _dx}[case["op"]](s, case)


def _masked(t, ids, L):
    """t [M, L, r], zero where the row's adapter is another."""
    hit = ids[:, None] == torch.arange(L, device=ids.device, dtype=ids.dtype)
    return torch.where(hit[:, :, None], t, torch.zeros((), device=t.device))


def _forward(s, case):
    """(y', h by adapter [M, L, r]) in 32 bits."""
    M, L, r = case["M"], case["L"], case["r"]
    A, B = s["A"].float(), s["B"].float()
    h = _masked((s["x"].float() @ A.view(L * r, -1).t()).view(M, L, r), s["ids"], L)
    y = s["y"].float() + (h * s["scale"][:, None]).view(M, L * r) @ B.view(L * r, -1)
    return y.to(torch.bfloat16), h


def _lora(s, case):
    if own:
        import gemm_any4_amd as any4

        return any4.lora(s["x"], s["A"], s["B"], s["scale"], s["ids"], s["y"], out=torch.empty_like(s["y"]))
    return _forward(s, case)[0]


def _codes8(x):
    """(whole numbers [M, K/128, 128], scales [M, K/128, 1]) of an activation.
    The quotients are taken in 64 bits: a scalar divided by a tensor is a
    product with the reciprocal, and one bit there moves values at a border
    between two whole numbers."""
    v = x.float().view(x.shape[0], -1, GROUP)
    amax = v.abs().amax(dim=2, keepdim=True).double()
    live = amax >= 2.0 ** -100
    inv = torch.where(live, 127.0 / amax, torch.zeros_like(amax)).float()
    return torch.round(v * inv), torch.where(live, amax / 127.0, torch.zeros_like(amax)).float()


def _train(s, case):
    M, L, r = case["M"], case["L"], case["r"]
    if own:
        import gemm_any4_amd as any4

        h = torch.empty((M, r), dtype=torch.float32, device=s["x"].device)
        x, x_scale, act = s["x"], None, None
        if case["act8"]:
            x, x_scale = act = any4.act8_empty(x)
        y = any4.lora(s["x"], s["A"], s["B"], s["scale"], s["ids"], s["y"], out=torch.empty_like(s["y"]), h=h, act=act)
        dx, dA, dB = any4.lora_backward(s["dy"], x, h, s["A"], s["B"], s["scale"], s["ids"], dx=s["dx"],
                                        out=torch.empty_like(s["dx"]), x_scale=x_scale)
        return {"y": y, "h": h, "dx": dx, "dA": dA, "dB": dB}
    y, h = _forward(s, case)
    x = s["x"].float()
    if case["act8"]:
        q, unit = _codes8(s["x"])
        x = (q * unit).view(M, -1)
    A, B, dy = s["A"].float().view(L * r, -1), s["B"].float().view(L * r, -1), s["dy"].float()
    dh = _masked((dy @ B.t()).view(M, L, r) * s["scale"][:, None], s["ids"], L).view(M, L * r)
    dx = (s["dx"].float() + dh @ A).to(torch.bfloat16)
    dA = (dh.t() @ x).view(L, r, -1)
    dB = ((h * s["scale"][:, None]).view(M, L * r).t() @ dy).view(L, r, -1)
    return {"y": y, "h": h.sum(dim=1), "dx": dx, "dA": dA, "dB": dB}


def _act8(s, case):
    if own:
        import gemm_any4_amd as any4

        return any4.act8_load(*any4.act8_save(s["x"]))
    q, unit = _codes8(s["x"])
    return (q * unit).view_as(s["x"]).to(torch.bfloat16)


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


def _dx(s, case):
    N, K, g = case["N"], case["K"], case["g"]
    if own:
        import gemm_any4_amd as any4

        if case["fmt"] == "int4":
            return any4.gemm_int4_dx(s["dy"], s["packed"], s["alpha"], s["beta"], g)
        call = {"any4": any4.gemm_dx, "any2": any4.any2_gemm_dx, "any3": any4.any3_gemm_dx}[case["fmt"]]
        return call(s["dy"], s["packed"], s["lut"], s["alpha"], s["beta"], g)
    code = _unpack(s["packed"], N, K, CODE_BITS[case["fmt"]])
    v = code.float() if case["fmt"] == "int4" else torch.gather(s["lut"].float(), 1, code.long())
    v = v.view(N, -1, g) * s["alpha"].float()[:, :, None] + s["beta"].float()[:, :, None]
    w = v.to(torch.bfloat16).float().view(N, K)      # a weight is a bf16 value
    return (s["dy"].float() @ w).to(torch.bfloat16)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "act8":
        return _exact_act8(s["x"])
    if op == "dx":
        return s["dy"].double() @ _exact_weights(s, case)
    x, y = s["x"].double(), s["y"].double()
    h = torch.zeros(case["M"], case["r"], dtype=torch.float64, device=x.device)
    dx, dy = (s["dx"].double(), s["dy"].double()) if op == "train" else (None, None)
    dA = torch.zeros(s["A"].shape, dtype=torch.float64, device=x.device)
    dB = torch.zeros(s["B"].shape, dtype=torch.float64, device=x.device)
    kept = _exact_act8(s["x"]) if case.get("act8") else x
    for a in range(case["L"]):
        rows = torch.nonzero(s["ids"] == a).flatten()
        Aa, Ba, sa = s["A"][a].double(), s["B"][a].double(), s["scale"][a].double()
        h[rows] = x[rows] @ Aa.t()
        y[rows] += sa * (h[rows] @ Ba)
        if op == "train":
            dh = sa * (dy[rows] @ Ba.t())
            dx[rows] += dh @ Aa
            dA[a] = dh.t() @ kept[rows]
            dB[a] = sa * (h[rows].t() @ dy[rows])
    return y if op == "lora" else {"y": y, "h": h, "dx": dx, "dA": dA, "dB": dB}


def _exact_act8(x):
    """An 8-bit activation's values: the scale and its inverse are defined as
    32-bit quotients and the scaled value as their product rounded to 32 bits;
    what follows is exact."""
    M, K = x.shape
    v = x.double().reshape(M * (K // GROUP), GROUP)
    top = v.abs().max(dim=1, keepdim=True).values
    unit, inv = (top / 127).float().double(), (127 / top).float().double()
    out = torch.round((v * inv).float().double()) * unit
    return torch.where(top < 2.0 ** -100, torch.zeros_like(out), out).view(M, K)


def _exact_weights(s, case):
    """W [N, K]: alpha * value + beta in 64 bits (exact but for far exponents),
    rounded to 32 bits and then to the bf16 that a weight is."""
    N, K, g, fmt = case["N"], case["K"], case["g"], case["fmt"]
    bits = CODE_BITS[fmt]
    n = torch.arange(N, device="cuda")[:, None]
    k = torch.arange(K, device="cuda")[None, :]
    # slot of 32 codes: row block, chunk of 128 k, quarter of it, row in the block
    slot = ((n // 16 * (K // 128) + k // 128) * 4 + k % 128 // 32) * 16 + n % 16
    i, size = k % 32, 4 * bits
    if bits == 3:
        p = i // 2
        low = s["packed"][slot * size + p.clamp(max=11)].long() & 63
        j = (p - 12).clamp(min=0)
        t = [s["packed"][slot * size + j + 4 * q].long() >> 6 << 2 * q for q in range(3)]
        code = torch.where(p < 12, low, t[0] + t[1] + t[2]) >> 3 * (i % 2) & 7
    else:
        per = 8 // bits
        code = s["packed"][slot * size + i // per].long() >> bits * (i % per) & (1 << bits) - 1
    value = code.double() if fmt == "int4" else s["lut"].double().gather(1, code)
    w = s["alpha"].double().repeat_interleave(g, 1) * value + s["beta"].double().repeat_interleave(g, 1)
    return w.float().to(torch.bfloat16).double()
