"""The expert operators a program composes itself: what is measured of them.

Products of ragged expert groups (``offsets`` as ``moe_permute`` writes them)
with each expert's matrix, forward and for both gradients; the same product in
8-bit integers with one scale per token and one per output channel, together
with the step that makes the integers; and SwiGLU with its gradient between
two products.

``run`` makes one pass: in plain torch operations (``own`` false) or through
the library (``own`` true).  Shapes are those of the repository's layer
configurations, or generic.
"""
import math

import torch
import torch.nn.functional as F

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}

# kinds of pass:
#   fwd     out[r] = x[r] W_e^T for the rows r of expert e
#   grad    dx[r] = dy[r] W_e and dW_e = sum over its rows of dy[r]^T x[r]
#   i8_up   tokens -> int8 rows in expert order -> int8 product (gate and up)
#   i8_down gate and up -> SwiGLU to int8 rows -> int8 product (down)
#   swiglu  h = silu(g) u, and the gradient of gate_up for a given dh


def _case(name, kind, T, k, E, N, K, type="bf16", out="bf16", zipf=0.0, idle=0):
    return {"name": name, "kind": kind, "tokens": T, "top_k": k, "experts": E, "N": N, "K": K, "type": type,
            "out": out, "zipf": zipf, "idle": idle}


def listed():
    return [
        # the tiny layer's gate/up product: nothing but latency
        _case("fwd_tiny", "fwd", 16, 2, 8, 1024, 256, "fp16", "fp16"),
        # one decoded token of the gpt-oss-shaped layer with bf16 experts: four
        # experts' weights are read for one row each
        _case("fwd_decode_T1", "fwd", 1, 4, 128, 5760, 2880),
        # the same layer's decode batch of 64: about two rows per expert, most experts touched
        _case("fwd_decode_T64", "fwd", 64, 4, 128, 5760, 2880),
        # Mixtral-shaped prefill, gate/up: compute bound, about 1024 rows per expert
        _case("fwd_prefill", "fwd", 4096, 2, 8, 28672, 4096),
        # a small odd training step in fp16: ragged groups, a third of the
        # experts without a row, sizes that fill no tile
        _case("grad_ragged", "grad", 523, 3, 24, 1100, 836, "fp16", "fp16", 1.1, 8),
        # gpt-oss-shaped down projection, training batch: 64 rows per expert on
        # average, weight gradients kept in fp32 (their write is the most traffic)
        _case("grad_fp32", "grad", 2048, 4, 128, 2880, 2880, "bf16", "fp32"),
        # Mixtral-shaped gate/up, both gradients: compute bound
        _case("grad_prefill", "grad", 4096, 2, 8, 28672, 4096),
        # one decoded token with int8 experts, gpt-oss-shaped gate/up
        _case("i8_up_decode_T1", "i8_up", 1, 4, 128, 5760, 2880),
        # Kimi-shaped decode batch, gate/up, Zipf-skewed routing over 384 experts
        _case("i8_up_decode_T128", "i8_up", 128, 8, 384, 4096, 7168, zipf=1.1),
        # Mixtral-shaped prefill, down projection in int8
        _case("i8_down_prefill", "i8_down", 4096, 2, 8, 4096, 14336),
        # SwiGLU between two products, a decode batch of the gpt-oss-shaped layer
        _case("swiglu_decode", "swiglu", 64, 4, 128, 0, 2880, "fp16", "fp16"),
        # SwiGLU and its gradient over a Mixtral-shaped training batch
        _case("swiglu_train", "swiglu", 4096, 2, 8, 0, 14336),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["fwd", "fwd", "grad", "grad", "i8_up", "i8_up", "i8_down", "swiglu"])
    while True:
        E = _log(rng, 1, 384)
        k = rng.randint(1, min(8, E))
        T = _log(rng, 1, 4096)
        N, K = _log(rng, 64, 28672), _log(rng, 64, 14336)
        if rng.random() < 0.5:  # half of the draws keep to multiples of 32, the rest are any size
            N, K = -(-N // 32) * 32, -(-K // 32) * 32
        if kind == "swiglu":
            N = 0
        if E * N * K <= 940e6 and T * k * N * K <= 0.9e12 and T * k * (2 * K if kind != "fwd" else K) <= 240e6:
            break
    t = rng.choice(["bf16", "fp16"])
    out = rng.choice([t, t, "fp32"]) if kind in ("fwd", "grad") else rng.choice(["bf16", "fp16", "fp32"])
    if kind == "swiglu":
        out = t
    idle = rng.randint(0, E - k) if rng.random() < 0.3 else 0
    c = _case("", kind, T, k, E, N, K, t, out, rng.choice([0.0, 0.0, 1.1]), idle)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _pitched(shape, dtype):
    """A tensor whose rows start on 16-byte boundaries, as the product's operands have to."""
    per = 16 // torch.empty(0, dtype=dtype).element_size()
    full = torch.zeros(*shape[:-1], -(-shape[-1] // per) * per, dtype=dtype, device=DEV)
    return full[..., : shape[-1]]


def _normal(shape, dtype, g, std=1.0):
    t = _pitched(shape, dtype)
    t.copy_(torch.empty(shape, dtype=dtype, device=DEV).normal_(0.0, std, generator=g))
    return t


def _route(c, g, device):
    """Experts of each token: k different ones by random scores, skewed and partly idle as the case says."""
    T, k, E = c["tokens"], c["top_k"], c["experts"]
    u = torch.rand(T, E, generator=g, device=device).clamp_(1e-7, 1 - 1e-7)
    score = -torch.log(-torch.log(u))
    rank = torch.randperm(E, generator=g, device=device).float() + 1
    score -= c["zipf"] * rank.log()
    score[:, torch.randperm(E, generator=g, device=device)[: c["idle"]]] = -math.inf
    return score.topk(k, dim=1).indices


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed)
    T, k, E, N, K = c["tokens"], c["top_k"], c["experts"], c["N"], c["K"]
    kind, t, ot = c["kind"], TYPES[c["type"]], TYPES[c["out"]]
    R = T * k
    s = {"kind": kind, "out_type": ot}
    if kind == "swiglu":
        s["gate_up"] = _normal((R, 2 * K), t, g)
        s["dh"] = _normal((R, K), t, g, 0.1)
        s["h"] = torch.empty(R, K, dtype=t, device=DEV)
        s["dgate_up"] = torch.empty(R, 2 * K, dtype=t, device=DEV)
        return s
    expert = _route(c, g, DEV).reshape(-1)
    order = torch.argsort(expert, stable=True)
    counts = torch.bincount(expert, minlength=E)
    s["row_token"] = (order // k).to(torch.int32)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    # where each row lies in a batch of equally long groups of the experts in use (the plain form's)
    s["used"] = counts.nonzero().squeeze(1)
    s["group"] = torch.searchsorted(s["used"], expert[order])
    s["place"] = torch.arange(R, device=DEV) - s["offsets"][expert[order]]
    s["cap"] = int(counts.max())
    s["experts"] = E
    if kind in ("fwd", "grad"):
        s["x"] = _normal((R, K), t, g)
        s["w"] = _pitched((E, N, K), t)
        for e in range(E):
            s["w"][e].copy_(torch.empty(N, K, dtype=t, device=DEV).normal_(0.0, 0.02, generator=g))
        if kind == "fwd":
            s["out"] = torch.empty(R, N, dtype=ot, device=DEV)
        else:
            s["dy"] = _normal((R, N), t, g, 0.1)
            s["dx"] = torch.empty(R, K, dtype=t, device=DEV)
            s["dw"] = torch.empty(E, N, K, dtype=ot, device=DEV)
        return s
    s["w"] = _pitched((E, N, K), torch.int8)
    for e in range(E):  # codes of normally distributed weights, the largest of a channel about four deviations out
        s["w"][e].copy_(torch.empty(N, K, device=DEV).normal_(0.0, 32.0, generator=g).round_().clamp_(-127, 127))
    s["w_scale"] = (0.5 + torch.rand(E, N, generator=g, device=DEV)) * (0.02 / 32.0)
    if kind == "i8_up":
        s["x"] = _normal((T, K), t, g)
    else:
        s["x"] = _normal((R, 2 * K), t, g)
    s["q"] = _pitched((R, K), torch.int8)
    s["q_scale"] = torch.empty(R, dtype=torch.float32, device=DEV)
    s["out"] = torch.empty(R, N, dtype=ot, device=DEV)
    return s


# -------------------------------------------------------------- plain forms

def _batched(s, rows):
    """Rows in expert order -> [experts in use][longest group][width], zeros behind each group."""
    b = rows.new_zeros(s["used"].numel(), s["cap"], rows.shape[1])
    b[s["group"], s["place"]] = rows
    return b


def _flat(s, b):
    return b[s["group"], s["place"]]


def _plain_fwd(s):
    w = s["w"][s["used"]].float()
    return _flat(s, torch.bmm(_batched(s, s["x"].float()), w.transpose(1, 2))).to(s["out_type"])


def _plain_grad(s):
    x, dy = _batched(s, s["x"].float()), _batched(s, s["dy"].float())
    dx = _flat(s, torch.bmm(dy, s["w"][s["used"]].float())).to(s["x"].dtype)
    dw = torch.zeros(s["w"].shape, dtype=s["out_type"], device=DEV)
    dw[s["used"]] = torch.bmm(dy.transpose(1, 2), x).to(s["out_type"])
    return {"dx": dx, "dw": dw}


def _silu_mul(gate_up):
    g, u = gate_up.float().chunk(2, dim=1)
    return g / (1 + torch.exp(-g)) * u


def _codes(v):
    """int8 codes and scale of each row: scale = amax / 127, code = round(v * (127 / amax)), each step rounded to fp32."""
    amax = v.abs().amax(dim=1, keepdim=True)
    none = amax < 2.0 ** -120
    top = torch.full_like(amax, 127.0)  # a tensor: a division by or of a plain number would go over a reciprocal
    q = torch.where(none, 0.0, torch.round(v * (top / amax)).clamp(-127, 127))
    return q, torch.where(none, 0.0, amax / top)


def _plain_i8(s):
    v = s["x"].float()[s["row_token"].long()] if s["kind"] == "i8_up" else _silu_mul(s["x"])
    q, scale = _codes(v)
    # the integer sums pass 2^24: in 64 bits
    acc = _flat(s, torch.bmm(_batched(s, q.double()), s["w"][s["used"]].double().transpose(1, 2)))
    return (acc * scale.double() * s["w_scale"][s["used"][s["group"]]].double()).to(s["out_type"])


def _plain_swiglu(s):
    g, u = s["gate_up"].float().chunk(2, dim=1)
    dh = s["dh"].float()
    sig = 1 / (1 + torch.exp(-g))
    silu = g * sig
    d = torch.cat([dh * u * sig * (1 + g * (1 - sig)), dh * silu], dim=1)
    return {"h": (silu * u).to(s["h"].dtype), "dgate_up": d.to(s["h"].dtype)}


def _own(s):
    import expert_ffn_layer_route_b200 as moe

    kind = s["kind"]
    if kind == "fwd":
        moe.moe_grouped_gemm(s["x"], s["w"], s["offsets"], s["out"])
        return s["out"]
    if kind == "grad":
        moe.moe_grouped_gemm_grad_x(s["dy"], s["w"], s["offsets"], s["dx"])
        moe.moe_grouped_gemm_grad_w(s["dy"], s["x"], s["offsets"], s["dw"])
        return {"dx": s["dx"], "dw": s["dw"]}
    if kind == "swiglu":
        moe.moe_swiglu(s["gate_up"], s["h"])
        moe.moe_swiglu_grad(s["gate_up"], s["dh"], s["dgate_up"])
        return {"h": s["h"], "dgate_up": s["dgate_up"]}
    if kind == "i8_up":
        moe.moe_quant_rows_i8(s["x"], s["q"], s["q_scale"], row_token=s["row_token"])
    else:
        moe.moe_swiglu_quant_i8(s["x"], s["q"], s["q_scale"])
    moe.moe_grouped_gemm_i8(s["q"], s["q_scale"], s["w"], s["w_scale"], s["offsets"], s["out"])
    return s["out"]


def run(state):
    if own:
        return _own(state)
    return {"fwd": _plain_fwd, "grad": _plain_grad, "i8_up": _plain_i8, "i8_down": _plain_i8,
            "swiglu": _plain_swiglu}[state["kind"]](state)


# --------------------------------------------------------------- accounting

def _experts_in_use(c):
    g = torch.Generator().manual_seed(1)
    return int(_route(c, g, "cpu").unique().numel())


def work(case):
    c = dict(case)
    T, R, E, N, K = c["tokens"], c["tokens"] * c["top_k"], c["experts"], c["N"], c["K"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    a, o = size[c["type"]], size[c["out"]]
    kind = c["kind"]
    if kind == "swiglu":
        # gate_up and dh read, h and dgate_up written; an exp, two divisions and about ten products a value
        return {"bytes": R * K * a * (2 + 1 + 1 + 2), "flops": R * K * 16}
    used = _experts_in_use(c)
    if kind == "fwd":
        return {"bytes": used * N * K * a + R * K * a + R * N * o, "flops": 2 * R * N * K}
    if kind == "grad":
        return {"bytes": used * N * K * a + R * (N + 2 * K) * a + E * N * K * o, "flops": 4 * R * N * K}
    x = T * K * a if kind == "i8_up" else R * 2 * K * a
    return {"bytes": x + used * N * (K + 4) + R * N * o, "flops": 2 * R * N * K}


# --------------------------------------------- the definition, in 64 bits

def _exact_codes(v):
    """The rule of the codes is stated in fp32 (two divisions and one product, each rounded once): followed as stated."""
    f = torch.float32
    amax = v.abs().max(dim=1).values
    live = amax >= 2.0 ** -120
    safe = torch.where(live, amax, torch.ones_like(amax))
    inv = (127.0 / safe).to(f).double()
    scale = (safe / 127.0).to(f).double()
    q = (v * inv[:, None]).to(f).double().round().clamp(-127, 127)
    return q * live[:, None], scale * live


def exact(case, seed):
    s = prepare(case, seed)
    kind = s["kind"]
    if kind == "swiglu":
        gu, dh = s["gate_up"].double(), s["dh"].double()
        K = dh.shape[1]
        g, u = gu[:, :K], gu[:, K:]
        sig = torch.sigmoid(g)
        slope = sig + g * sig * (1 - sig)
        return {"h": g * sig * u, "dgate_up": torch.cat([dh * u * slope, dh * g * sig], dim=1)}
    at = s["offsets"].tolist()
    w = s["w"]
    E, N, K = w.shape
    R = at[-1]
    if kind == "grad":
        dx = torch.empty(R, K, dtype=torch.float64, device=DEV)
        dw = torch.zeros(E, N, K, dtype=torch.float64, device=DEV)
    else:
        out = torch.empty(R, N, dtype=torch.float64, device=DEV)
    for e in range(E):
        rows = slice(at[e], at[e + 1])
        if at[e] == at[e + 1]:
            continue
        we = w[e].double()
        if kind == "fwd":
            out[rows] = s["x"][rows].double() @ we.t()
        elif kind == "grad":
            dy = s["dy"][rows].double()
            dx[rows] = dy @ we
            dw[e] = dy.t() @ s["x"][rows].double()
        else:
            if kind == "i8_up":
                v = s["x"][s["row_token"][rows].long()].double()
            else:
                g, u = s["x"][rows, :K].double(), s["x"][rows, K:].double()
                v = g * torch.sigmoid(g) * u
            q, scale = _exact_codes(v)
            out[rows] = (q @ we.t()) * scale[:, None] * s["w_scale"][e].double()[None, :]
    return {"dx": dx, "dw": dw} if kind == "grad" else out
