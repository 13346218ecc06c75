"""Cases for three operators of a mixture-of-experts layer in 8-bit floating point.

linear   Y = X W^T with E4M3 operands: a weight scale for each 128 x 128 block, an activation
         scale for each token and 128 channels, found from X within the call.
route    router logits -> the top-k experts of each token and their weights (softmax or sigmoid
         scores, a balance bias, groups, renormalisation).
experts  the routed feed-forward: Y[t] = sum_j w[t,j] * down_e(silu(gate_e(x_t)) * up_e(x_t)),
         e = ids[t,j]; x_t and the hidden vectors are E4M3 with a scale per token and 128 channels.

``own`` selects between the plain torch form (False) and the library's kernels (True).
"""
import math

import torch

own = False
fmpq = None    # the library's binding, imported where its kernels are called
BLOCK = 128
QMAX = 448.0   # largest E4M3 value


def _library():
    global fmpq
    if fmpq is None:
        from bit_quantized_gemm_fmpq_gb300 import fmpq as lib
        fmpq = lib
    return fmpq


# ------------------------------------------------------------------------------ the cases

def listed():
    return [
        # one token of a 70B-class square projection (the decode sweep's layer): latency, weight stream
        dict(name="linear_one_token", op="linear", M=1, K=8192, N=8192, dtype="float16", pad=0),
        # a decode batch on the same layer: still the weight stream
        dict(name="linear_decode_batch", op="linear", M=32, K=8192, N=8192, dtype="bfloat16", pad=0),
        # a prompt through the QKV projection of a 7B-class model
        dict(name="linear_qkv_prompt", op="linear", M=2048, K=4096, N=12288, dtype="bfloat16", pad=0),
        # odd everything, rows with a stride: a batch of leftovers through an unaligned layer
        dict(name="linear_ragged", op="linear", M=515, K=2868, N=4004, dtype="float16", pad=12),
        # the gate/up projection of a 70B-class model, 4096 tokens: the largest product
        dict(name="linear_gate_up", op="linear", M=4096, K=8192, N=28672, dtype="bfloat16", pad=0),
        # one token's routing: pure latency
        dict(name="route_one_token", op="route", T=1, E=64, k=6, dtype="bfloat16", score="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renormalize=True, scale=1.0, masked=0.0),
        # a long prompt, many experts, sigmoid scores with a balance bias, limited to 4 of 8 groups
        dict(name="route_prompt_groups", op="route", T=16384, E=256, k=8, dtype="float32", score="sigmoid", bias=True,
             groups=8, top_groups=4, group_top=2, renormalize=True, scale=2.5, masked=0.0),
        # an odd expert count, experts masked out by -inf, padding tokens with every expert masked
        dict(name="route_ragged_masked", op="route", T=4099, E=60, k=4, dtype="bfloat16", score="softmax", bias=False,
             groups=1, top_groups=1, group_top=1, renormalize=False, scale=1.0, masked=0.1),
        # one token through its 8 experts of 128: latency, the weights of 8 experts
        dict(name="experts_one_token", op="experts", T=1, E=128, k=8, H=4096, F=1024, dtype="bfloat16", skew=0.0,
             dropped=0.0),
        # a decode batch: nearly every expert is read for a few tokens each
        dict(name="experts_decode_batch", op="experts", T=64, E=128, k=8, H=4096, F=1024, dtype="bfloat16", skew=0.0,
             dropped=0.0),
        # a prompt: 256 tokens an expert on average
        dict(name="experts_prompt", op="experts", T=4096, E=128, k=8, H=4096, F=1024, dtype="bfloat16", skew=0.0,
             dropped=0.0),
        # few experts, odd sizes, an uneven load, some slots without an expert
        dict(name="experts_ragged", op="experts", T=777, E=10, k=2, H=2012, F=1404, dtype="float16", skew=1.0,
             dropped=0.05),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "route", "experts", "experts"])
    dtype = rng.choice(["float16", "bfloat16"])
    if op == "linear":
        while True:
            c = dict(op="linear", M=_log_int(rng, 1, 8192), K=_log_int(rng, 100, 16384), N=_log_int(rng, 100, 28672),
                     dtype=dtype, pad=rng.choice([0, 0, 1, 8]))
            if rng.random() < 0.5:   # widths of real layers are mostly multiples of 128
                c["K"], c["N"] = max(128, c["K"] // 128 * 128), max(128, c["N"] // 128 * 128)
            if c["M"] * c["K"] * c["N"] <= 4096 * 8192 * 28672 and 3072 not in (c["M"], c["K"], c["N"]):
                return c
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _log_int(rng, 4, 512 // groups // 2)
        k = rng.randint(1, min(8, E))
        top_groups = rng.randint(1, groups)
        while top_groups * (E // groups) < k:
            top_groups += 1
        bias = rng.random() < 0.5
        return dict(op="route", T=_log_int(rng, 1, 16384), E=E, k=k, dtype=rng.choice(["float32", "bfloat16", "float16"]),
                    score=rng.choice(["softmax", "sigmoid"]), bias=bias, groups=groups, top_groups=top_groups,
                    group_top=2 if bias else 1, renormalize=rng.random() < 0.7, scale=rng.choice([1.0, 2.5]),
                    masked=rng.choice([0.0, 0.1]))
    while True:
        E = rng.randint(2, 128)
        c = dict(op="experts", T=_log_int(rng, 1, 4096), E=E, k=rng.randint(1, min(8, E)), H=_log_int(rng, 256, 8192),
                 F=_log_int(rng, 128, 4096), dtype=dtype, skew=rng.choice([0.0, 0.5, 1.0]),
                 dropped=rng.choice([0.0, 0.05]))
        if rng.random() < 0.5:
            c["H"], c["F"] = c["H"] // 128 * 128, c["F"] // 128 * 128
        if (c["T"] * c["k"] * c["H"] * c["F"] <= 4096 * 8 * 4096 * 1024 and E * c["H"] * c["F"] <= 128 * 4096 * 1024
                and 3072 not in (c["T"], c["H"], c["F"], 2 * c["F"])):
            return c


def work(case):
    if case["op"] == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        scales = -(-N // BLOCK) * -(-K // BLOCK) * 4
        return {"bytes": 2 * M * K + N * K + scales + 2 * M * N, "flops": 2.0 * M * N * K}
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["k"]
        size = 4 if case["dtype"] == "float32" else 2
        # per logit: a score (an exponential counted as 8) and k compares
        return {"bytes": T * E * size + (4 * E if case["bias"] else 0) + 8 * T * k, "flops": float(T * E * (8 + k))}
    T, E, k, H, F = case["T"], case["E"], case["k"], case["H"], case["F"]
    hit = E * (1.0 - (1.0 - k / E) ** T)   # experts that some token uses, on average
    return {"bytes": int(hit * 3 * H * F * (1 + 4 / BLOCK ** 2)) + 2 * 2 * T * H + 8 * T * k,
            "flops": 2.0 * T * k * 3 * H * F * (1.0 - case["dropped"])}


# ------------------------------------------------------------------------------ the inputs

def _generator(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1000003 * seed + 17)
    return g


def _checkpoint(g, N, K, std):
    """One E4M3 weight matrix [N, K] with its 128 x 128 block scales: values of about N(0, std^2)."""
    codes = torch.randn(N, K, generator=g, device="cuda").mul_(120.0).clamp_(-QMAX, QMAX).to(torch.float8_e4m3fn)
    scales = torch.rand(-(-N // BLOCK), -(-K // BLOCK), generator=g, device="cuda").add_(0.5).mul_(std / 120.0)
    return codes, scales


def prepare(case, seed):
    g = _generator(case, seed)
    op = case["op"]
    dtype = getattr(torch, case["dtype"])
    st = dict(case=case)
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        # N(0, 1) activations with 10 % of the channels larger by 20 to 100 (outlier channels)
        amp = torch.ones(K, device="cuda")
        loud = torch.rand(K, generator=g, device="cuda") < 0.1
        amp = torch.where(loud, torch.rand(K, generator=g, device="cuda") * 80 + 20, amp)
        X = torch.empty(M, K + case["pad"], dtype=dtype, device="cuda")[:, :K]
        X.copy_(torch.randn(M, K, generator=g, device="cuda") * amp)
        st["X"] = X
        codes, scales = _checkpoint(g, N, K, 0.02)
        if own:
            lib = _library()
            st["layer"] = lib.Fp8Layer(K, N)
            st["W"] = lib.fp8_pack_codes(st["layer"], codes, scales)
        else:
            st["W"] = (codes, scales)
        return st
    if op == "route":
        T, E = case["T"], case["E"]
        logits = torch.randn(T, E, generator=g, device="cuda") * 1.5
        if case["masked"] > 0:
            off = torch.rand(T, E, generator=g, device="cuda") < case["masked"]
            off |= torch.rand(T, 1, generator=g, device="cuda") < case["masked"] / 4   # padding tokens
            logits = logits.masked_fill(off, float("-inf"))
        st["logits"] = logits.to(dtype)
        st["bias"] = torch.randn(E, generator=g, device="cuda") * 0.05 if case["bias"] else None
        if own:
            _library()
        return st
    T, E, k, H, F = case["T"], case["E"], case["k"], case["H"], case["F"]
    st["X"] = torch.randn(T, H, generator=g, device="cuda").to(dtype)
    load = torch.rand(E, generator=g, device="cuda") * 2 * case["skew"]      # some experts are liked better
    liking = load - torch.rand(T, E, generator=g, device="cuda").clamp_min(1e-9).log().neg().log()
    ids = liking.topk(k, dim=1).indices.to(torch.int32)
    weights = torch.rand(T, k, generator=g, device="cuda") + 0.2
    weights = weights / weights.sum(1, keepdim=True)
    gone = torch.rand(T, k, generator=g, device="cuda") < case["dropped"]
    st["ids"] = ids.masked_fill(gone, -1)
    st["weights"] = weights.masked_fill(gone, 0.0)
    up_codes, up_scales, down_codes, down_scales = [], [], [], []
    for _ in range(E):
        gate = _checkpoint(g, F, H, 1.0 / math.sqrt(H))
        up = _checkpoint(g, F, H, 1.0 / math.sqrt(H))
        down = _checkpoint(g, H, F, 1.0 / math.sqrt(F))
        up_codes.append(torch.cat([gate[0].view(torch.uint8), up[0].view(torch.uint8)]))
        up_scales.append(torch.cat([gate[1], up[1]]))
        down_codes.append(down[0].view(torch.uint8))
        down_scales.append(down[1])
    up_codes = torch.stack(up_codes).view(torch.float8_e4m3fn)         # [E, 2F, H]: gate rows, then up rows
    down_codes = torch.stack(down_codes).view(torch.float8_e4m3fn)     # [E, H, F]
    up_scales, down_scales = torch.stack(up_scales), torch.stack(down_scales)
    if own:
        lib = _library()
        st["up"] = lib.Fp8Layer(H, 2 * F, experts=E, gated=True)
        st["down"] = lib.Fp8Layer(F, H, experts=E)
        st["W_up"] = lib.fp8_pack_codes(st["up"], up_codes, up_scales)
        st["W_down"] = lib.fp8_pack_codes(st["down"], down_codes, down_scales)
    else:
        st["W_up"], st["W_down"] = (up_codes, up_scales), (down_codes, down_scales)
    return st


# ------------------------------------------------------------------------------ the plain forms

def _quantized(x):
    """The values that x stands for in E4M3 with a scale for each row and 128 channels (fp32)."""
    rows, K = x.shape
    pad = -K % BLOCK
    b = torch.nn.functional.pad(x.float(), (0, pad)).view(rows, -1, BLOCK)
    amax = b.abs().amax(2, keepdim=True)
    scale = amax / torch.full_like(amax, QMAX)
    codes = torch.where(scale > 0, b / scale, torch.zeros_like(b)).clamp(-QMAX, QMAX).to(torch.float8_e4m3fn)
    return (codes.float() * scale).view(rows, -1)[:, :K]


def _dequantized(codes, scales):
    N, K = codes.shape
    return codes.float() * scales.repeat_interleave(BLOCK, 0)[:N].repeat_interleave(BLOCK, 1)[:, :K]


def _plain_linear(st):
    X = st["X"]
    return (_quantized(X) @ _dequantized(*st["W"]).t()).to(X.dtype)


def _plain_route(st):
    c, logits, bias = st["case"], st["logits"], st["bias"]
    T, E, k = c["T"], c["E"], c["k"]
    x = logits.float()
    masked = x == float("-inf")
    top = x.amax(1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    if c["score"] == "softmax":
        e = torch.exp(x - top)
        total = e.sum(1, keepdim=True)
        score = e / torch.where(total > 0, total, torch.ones_like(total))
    else:
        score = 1.0 / (1.0 + torch.exp(-x))
    if bias is None and (c["groups"] == 1 or c["group_top"] == 1):
        key = x                       # both scores grow with the logit
    else:                             # close calls between biased scores: in 64 bits
        if c["score"] == "softmax":
            d = torch.exp(x.double() - top.double())
            t = d.sum(1, keepdim=True)
            key = d / torch.where(t > 0, t, torch.ones_like(t))
        else:
            key = 1.0 / (1.0 + torch.exp(-x.double()))
        if bias is not None:
            key = key + bias.double()
        key = key.masked_fill(masked, float("-inf"))
    if c["groups"] > 1:
        per = key.view(T, c["groups"], E // c["groups"])
        best = per.sort(dim=2, descending=True).values[:, :, :c["group_top"]]
        value = torch.where(best == float("-inf"), torch.zeros_like(best), best).sum(2)
        value = torch.where(best[:, :, 0] == float("-inf"), best[:, :, 0], value)
        order = value.sort(dim=1, descending=True, stable=True).indices[:, :c["top_groups"]]
        keep = torch.zeros(T, c["groups"], dtype=torch.bool, device=x.device).scatter_(1, order, True)
        key = per.masked_fill(~keep[:, :, None], float("-inf")).view(T, E)
    order = key.sort(dim=1, descending=True, stable=True)
    ids, none = order.indices[:, :k], order.values[:, :k] == float("-inf")
    w = score.gather(1, ids).masked_fill(none, 0.0)
    if c["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    return ids.to(torch.int32).masked_fill(none, -1), w * c["scale"]


def _plain_experts(st):
    X, ids, weights = st["X"], st["ids"], st["weights"]
    (uc, us), (dc, ds) = st["W_up"], st["W_down"]
    F = uc.shape[1] // 2
    half = us.shape[1] // 2
    out = torch.zeros(X.shape, dtype=torch.float32, device=X.device)
    xq = _quantized(X)
    for e in ids.unique().tolist():
        if e < 0:
            continue
        t, j = (ids == e).nonzero(as_tuple=True)
        x = xq[t]
        gate = x @ _dequantized(uc[e, :F], us[e, :half]).t()
        up = x @ _dequantized(uc[e, F:], us[e, half:]).t()
        h = gate / (1.0 + torch.exp(-gate)) * up
        out.index_add_(0, t, (_quantized(h) @ _dequantized(dc[e], ds[e]).t()) * weights[t, j, None])
    return out.to(X.dtype)


# ------------------------------------------------------------------------------ one pass

def run(state):
    c = state["case"]
    if not own:
        return {"linear": _plain_linear, "route": _plain_route, "experts": _plain_experts}[c["op"]](state)
    if c["op"] == "linear":
        return fmpq.fp8_quantize_gemm(state["layer"], state["X"], *state["W"])
    if c["op"] == "route":
        return fmpq.moe_route(state["logits"], c["k"], score=c["score"], bias=state["bias"], groups=c["groups"],
                              top_groups=c["top_groups"], group_top=c["group_top"], renormalize=c["renormalize"],
                              scale=c["scale"])
    return fmpq.moe_experts(state["up"], state["down"], state["X"], state["ids"], state["weights"], *state["W_up"],
                            *state["W_down"])


# ------------------------------------------------------------------------------ in 64 bits

def _e4m3_64(v):
    """Round to E4M3 (four significant bits, smallest step 2^-9, at most 448), ties to even."""
    mag = v.abs()
    exponent = torch.frexp(mag).exponent.double() - 1
    step = torch.exp2(exponent.clamp_min(-6.0) - 3)
    return torch.sign(v) * (torch.round(mag / step) * step).clamp_max(QMAX)


def _quantized_64(x):
    x = x.double()
    out = torch.empty_like(x)
    for lo in range(0, x.shape[1], BLOCK):
        v = x[:, lo:lo + BLOCK].float().double()
        s = (v.abs().max(1, keepdim=True).values / QMAX).float().double()   # scales and quotients are fp32
        q = (v / torch.where(s > 0, s, torch.ones_like(s))).float().double()
        out[:, lo:lo + BLOCK] = _e4m3_64(q) * s
    return out


def _weights_64(codes, scales):
    w = codes.float().double()
    rows = torch.arange(w.shape[0], device=w.device) // BLOCK
    cols = torch.arange(w.shape[1], device=w.device) // BLOCK
    return w.mul_(scales.double()[rows][:, cols])


def exact(case, seed):
    global own
    kept, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = kept
    if case["op"] == "linear":
        codes, scales = st["W"]
        if case["M"] * case["K"] * case["N"] > 4e12:
            return None
        x = _quantized_64(st["X"])
        y = torch.empty(case["M"], case["N"], dtype=torch.float64, device="cuda")
        for lo in range(0, case["N"], 4096):   # whole scale blocks at a time
            w = _weights_64(codes[lo:lo + 4096], scales[lo // BLOCK:(lo + 4096) // BLOCK])
            y[:, lo:lo + 4096] = x @ w.t()
        return y
    if case["op"] == "route":
        if case["T"] * case["k"] > 200000:
            return None
        x = st["logits"].double()
        open_ = x > float("-inf")
        if case["score"] == "softmax":
            score = torch.nan_to_num(torch.softmax(x, 1), nan=0.0)
        else:
            score = torch.sigmoid(x)
        plain_keys = st["bias"] is None and (case["groups"] == 1 or case["group_top"] == 1)
        key = x.clone() if plain_keys else score + (0.0 if st["bias"] is None else st["bias"].double())
        key[~open_] = float("-inf")
        T, E, n = case["T"], case["E"], case["groups"]
        if n > 1:
            blocks, value = key.view(T, n, E // n).clone(), torch.zeros(T, n, dtype=torch.float64, device="cuda")
            dead = blocks.amax(2) == float("-inf")
            left = blocks.clone()
            for _ in range(case["group_top"]):
                m, at = left.max(2, keepdim=True)
                value += torch.where(m == float("-inf"), torch.zeros_like(m), m)[:, :, 0]
                left.scatter_(2, at, float("-inf"))
            value[dead] = float("-inf")
            chosen = torch.zeros(T, n, dtype=torch.bool, device="cuda")
            for _ in range(case["top_groups"]):
                at = _first_max(value.masked_fill(chosen, float("-inf")), chosen)
                chosen[torch.arange(T, device="cuda"), at] = True
            key = blocks.masked_fill(~chosen[:, :, None], float("-inf")).view(T, E)
        ids = torch.empty(T, case["k"], dtype=torch.int32, device="cuda")
        w = torch.zeros(T, case["k"], dtype=torch.float64, device="cuda")
        row = torch.arange(T, device="cuda")
        for j in range(case["k"]):
            at = _first_max(key)
            some = key[row, at] > float("-inf")
            ids[:, j] = torch.where(some, at, torch.full_like(at, -1)).int()
            w[:, j] = torch.where(some, score[row, at], torch.zeros_like(w[:, j]))
            key[row, at] = float("-inf")
        if case["renormalize"]:
            total = w.sum(1, keepdim=True)
            w = torch.where(total > 0, w / total, torch.zeros_like(w))
        return ids, w * case["scale"]
    (uc, us), (dc, ds) = st["W_up"], st["W_down"]
    T, k, H, F = case["T"], case["k"], case["H"], case["F"]
    if 6.0 * T * k * H * F > 4e12:
        return None
    xq = _quantized_64(st["X"])
    y = torch.zeros(T, H, dtype=torch.float64, device="cuda")
    half = us.shape[1] // 2
    for e in range(case["E"]):
        for j in range(k):
            t = (st["ids"][:, j] == e).nonzero()[:, 0]
            if t.numel() == 0:
                continue
            g = xq[t] @ _weights_64(uc[e, :F], us[e, :half]).t()
            u = xq[t] @ _weights_64(uc[e, F:], us[e, half:]).t()
            h = _quantized_64(g * torch.sigmoid(g) * u)
            y[t] += st["weights"][t, j].double()[:, None] * (h @ _weights_64(dc[e], ds[e]).t())
    return y


def _first_max(v, taken=None):
    """Index of the largest entry of each row, the lowest such index (not one already taken)."""
    hit = v == v.amax(1, keepdim=True)
    if taken is not None:
        hit &= ~taken
        hit[hit.sum(1) == 0] = ~taken[hit.sum(1) == 0]
    place = torch.arange(v.shape[1], device=v.device)
    return torch.where(hit, place, torch.full_like(place, v.shape[1])).amin(1)
