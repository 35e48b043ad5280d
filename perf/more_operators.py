"""Workloads of the bf16 experts of a latent-MoE block, for prefill and training.

Five operators:

* ``gated``: both projections of a gated feed-forward block, the activation and
  the product in one pass, for rows sorted by expert or for one dense block (the
  shared expert); optionally with both projections kept for the backward pass, in
  bf16 or in 8 bits.
* ``gated_backward``: the gradients of its rows and weights from the projections
  that were kept, and the product again (the next projection's gradient needs it).
* ``matmul``, ``matmul_backward``: the product with the second weight of the block,
  and its gradients.
* ``checkpoint8``: activations written in 8 bits with one power of two per 16
  columns, and read back.

``prepare`` draws the inputs from the seed, ``run`` computes one pass, either
in plain torch operations (``own = False``) or through the package's entry
points, ``exact`` evaluates the definitions in 64 bits.

Shapes: 2048 latent columns, 7168 hidden columns, 1448 and 5128 columns, 16, 8192
and 16384 tokens, 256, 64 and 60 experts are those of this repository's benchmark
and of ``operators.py``; feed-forward widths are generic.
"""

import math

import torch

own = False

GROUP = 16  # columns that share a power of two


# ------------------------------------------------------------------ cases
def listed():
    return [
        # The shared expert of one decoded token: latency, the weights are read once.
        dict(name="gated_dense_T1", op="gated", T=1, K=1, E=1, C=7168, F=2048, drop=0.0, skew=0.0,
             save="none", act="silu"),
        # A decode step of 16 sequences: about 100 of 256 experts, one or two rows each.
        dict(name="gated_experts_T16", op="gated", T=16, K=8, E=256, C=2048, F=1024, drop=0.0,
             skew=0.0, save="none", act="silu"),
        # The shared expert of a prefill batch.
        dict(name="gated_dense_T8192", op="gated", T=8192, K=1, E=1, C=7168, F=2048, drop=0.0,
             skew=0.0, save="none", act="silu"),
        # Training on a ragged batch of a small model: odd counts and widths, some choices
        # without an expert, the projections kept in 8 bits.
        dict(name="gated_train_T1013", op="gated", T=1013, K=6, E=60, C=1448, F=712, drop=0.1,
             skew=1.0, save="8bit", act="gelu"),
        # A dense block on an odd batch with the projections kept in 8 bits.
        dict(name="gated_backward_T777", op="gated_backward", T=777, K=1, E=1, C=5128, F=1000,
             drop=0.0, skew=0.0, save="8bit", act="silu"),
        # Training of unevenly loaded experts.
        dict(name="gated_backward_T8192", op="gated_backward", T=8192, K=8, E=64, C=2048, F=1024,
             drop=0.0, skew=1.0, save="8bit", act="silu"),
        # The second projection of the decode step.
        dict(name="matmul_experts_T16", op="matmul", T=16, K=8, E=256, C=1024, M=2048, drop=0.0,
             skew=0.0),
        # The second projection of the largest prefill batch.
        dict(name="matmul_experts_T16384", op="matmul", T=16384, K=8, E=64, C=1024, M=2048,
             drop=0.0, skew=1.0),
        # Its gradients on the ragged batch.
        dict(name="matmul_backward_T1013", op="matmul_backward", T=1013, K=6, E=60, C=712, M=1448,
             drop=0.1, skew=1.0),
        # Its gradients in the shared expert.
        dict(name="matmul_backward_T4096", op="matmul_backward", T=4096, K=1, E=1, C=2048, M=7168,
             drop=0.0, skew=0.0),
        # One step's activations of 16 sequences: latency.
        dict(name="checkpoint8_T16", op="checkpoint8", T=16, C=7168),
        # A training batch's activations.
        dict(name="checkpoint8_T16384", op="checkpoint8", T=16384, C=7168),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["gated", "gated", "gated_backward", "matmul", "matmul_backward",
                     "checkpoint8"])
    if op == "checkpoint8":
        T = _log(rng, 1, 16384)
        return dict(op=op, T=T, C=8 * _log(rng, 8, min(2048, 16384 * 7168 // (8 * T))))
    if rng.random() < 0.4:
        T, K, E, drop, skew = _log(rng, 1, 8192), 1, 1, 0.0, 0.0
        C, wide = 8 * _log(rng, 16, 896), 8 * _log(rng, 16, 512)
    else:
        T, K, E = _log(rng, 1, 8192), rng.randint(1, 8), _log(rng, 8, 256)
        drop, skew = rng.choice([0.0, 0.0, 0.1, 0.4]), round(rng.uniform(0.0, 1.2), 2)
        C, wide = 8 * _log(rng, 16, 256), 8 * _log(rng, 16, 256)
        wide = max(128, min(wide, 8 * (128 * 2048 * 2048 // (8 * E * C))))
    passes = 2 if op.endswith("backward") else 1
    T = max(1, min(T, (8192 * 8192 * 2048) // (passes * K * C * wide)))
    case = dict(op=op, T=T, K=K, E=E, C=C, drop=drop, skew=skew)
    if op in ("matmul", "matmul_backward"):
        case["M"] = wide
        return case
    case["F"] = 8 * max(8, wide // 16)
    case["act"] = rng.choice(["silu", "silu", "gelu"])
    case["save"] = rng.choice(["bf16", "8bit", "8bit"] if op == "gated_backward" else
                              ["none", "none", "bf16", "8bit"])
    return case


# ----------------------------------------------------------------- inputs
def prepare(case, seed):
    dev, bf16 = torch.device("cuda"), torch.bfloat16
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    op, T, C = case["op"], case["T"], case["C"]

    def normal(*shape, scale=1.0):
        return torch.empty(*shape, dtype=bf16, device=dev).normal_(generator=gen).mul_(scale)

    if op == "checkpoint8":
        # Channels of unlike size, as activations have them.
        size = torch.exp(torch.randn(C, generator=gen, device=dev)).to(bf16)
        return dict(op=op, x=normal(T, C).mul_(size),
                    values=torch.empty(T, C, dtype=torch.int8, device=dev),
                    exponents=torch.empty(T, -(-C // GROUP), dtype=torch.uint8, device=dev),
                    out=torch.empty(T, C, dtype=bf16, device=dev))
    K, E = case["K"], case["E"]
    n, offsets, cap = T * K, None, T
    if E > 1:
        logits = torch.randn(T, E, generator=gen, device=dev)
        logits += case["skew"] * torch.randn(E, generator=gen, device=dev)
        ids = logits.topk(K, dim=1).indices
        routed = torch.rand(T, K, generator=gen, device=dev) >= case["drop"]
        counts = torch.bincount(ids[routed], minlength=E)
        cap = max(1, int(counts.max()))  # rows of the fullest expert
        offsets = torch.zeros(E + 1, dtype=torch.int32, device=dev)
        offsets[1:] = counts.cumsum(0)
    s = dict(op=op, offsets=offsets, cap=cap)

    def rows(width):
        """Rows in expert order; those past the last expert's are zero."""
        got = normal(n, width)
        if offsets is not None:
            got[torch.arange(n, device=dev) >= offsets[-1]] = 0
        return got

    s["x"] = rows(C)
    if op in ("matmul", "matmul_backward"):
        M = case["M"]
        s["weights"] = normal(E, M, C, scale=1 / math.sqrt(C))
        if op == "matmul":
            s["out"] = torch.empty(n, M, dtype=bf16, device=dev)
            return s
        s.update(grad_out=rows(M), grad_x=torch.empty_like(s["x"]),
                 grad_weights=torch.empty_like(s["weights"]))
        return s
    F, save = case["F"], case["save"]
    s.update(weights=normal(E, 2 * F, C, scale=1 / math.sqrt(C)), act=case["act"], save=save,
             hidden=torch.empty(n, F, dtype=bf16, device=dev))
    if op == "gated":
        s["saved"] = None
        if save == "bf16":
            s["saved"] = torch.empty(n, 2, F, dtype=bf16, device=dev)
        elif save == "8bit":
            s["saved"] = (torch.empty(n, 2, F, dtype=torch.int8, device=dev),
                          torch.empty(n, 2, -(-F // GROUP), dtype=torch.uint8, device=dev))
        return s
    # The backward pass has the forward's projections at hand, as they were kept.
    kept = rows(2 * F).unflatten(1, (2, F))
    s.update(saved=_pack8(kept) if save == "8bit" else kept, grad_hidden=rows(F),
             grad_x=torch.empty_like(s["x"]), grad_weights=torch.empty_like(s["weights"]),
             workspace=torch.empty(max(256, 4 * n * F), dtype=torch.uint8, device=dev))
    return s


# ------------------------------------------------------------ plain forms
def _grouped(v):
    """[..., C] in 32 bits as [..., groups, 16], zero behind the last column."""
    v = v.float()
    return torch.nn.functional.pad(v, (0, -v.shape[-1] % GROUP)).unflatten(-1, (-1, GROUP))


def _pack8(v):
    """(values, exponents): per 16 columns the least e >= 1 with round(max|v| / 2^(e-127)) <= 127,
    values round(v / 2^(e-127)); e = 0 for a group of zeros, 255 for one that is not finite."""
    g = _grouped(v)
    top = g.abs().amax(-1)
    mantissa, power = torch.frexp(top)            # top = mantissa * 2^power, 0.5 <= mantissa < 1
    e = power - 7 + (mantissa * 128 >= 127.5).to(power.dtype) + 127
    e = e.clamp(min=1)
    finite = torch.isfinite(g).all(-1)
    e = torch.where(finite, torch.where(top > 0, e, torch.zeros_like(e)), torch.full_like(e, 255))
    live = (finite & (top > 0))[..., None]
    q = torch.where(live, torch.ldexp(g, 127 - e[..., None]), torch.zeros_like(g)).round()
    return (q.to(torch.int8).flatten(-2)[..., :v.shape[-1]].contiguous(), e.to(torch.uint8))


def _unpack8(values, exponents):
    e = exponents.to(torch.int32)[..., None]
    v = torch.ldexp(_grouped(values), e - 127)
    v = torch.where(e == 255, torch.full_like(v, math.nan), v)
    return v.flatten(-2)[..., :values.shape[-1]]


def _sigma(g, act):
    """The factor s(g) of the activation g * s(g), and its derivative."""
    if act == "silu":
        s = torch.sigmoid(g)
        return s, s * (1 - s)
    k = math.sqrt(8 / math.pi)
    s = torch.sigmoid(k * (g + 0.044715 * g * g * g))
    return s, s * (1 - s) * k * (1 + 3 * 0.044715 * g * g)


def _spread(s, rows):
    """Rows of each expert, [E, cap, width] in 32 bits, zero behind the last."""
    if s["offsets"] is None:
        return rows.float()[None]
    at = s["offsets"][:-1, None].long() + torch.arange(s["cap"], device=rows.device)
    got = rows[at.clamp(max=rows.shape[0] - 1)].float()
    return got.masked_fill((at >= s["offsets"][1:, None])[..., None], 0.0)


def _back(s, spread, n):
    """The rows of ``_spread`` in their order, zero for rows without an expert."""
    if s["offsets"] is None:
        return spread[0]
    offsets = s["offsets"].long()
    r = torch.arange(n, device=spread.device)
    e = torch.searchsorted(offsets[1:], r, right=True).clamp(max=spread.shape[0] - 1)
    got = spread[e, (r - offsets[e]).clamp(0, spread.shape[1] - 1)]
    return got.masked_fill((r >= offsets[-1])[:, None], 0.0)


def _plain_matmul(s, x, w):
    return _back(s, torch.bmm(_spread(s, x), w.float().transpose(1, 2)), x.shape[0])


def _plain_matmul_backward(s, grad, x, w):
    g = _spread(s, grad)
    return (_back(s, torch.bmm(g, w.float()), x.shape[0]).to(x.dtype),
            torch.bmm(g.transpose(1, 2), _spread(s, x)).to(w.dtype))


def _plain_gated(s):
    pre = _plain_matmul(s, s["x"], s["weights"])
    gate, up = pre.chunk(2, dim=1)
    hidden = (gate * _sigma(gate, s["act"])[0] * up).to(s["x"].dtype)
    pre = pre.unflatten(1, (2, -1))
    if s["save"] == "none":
        return hidden
    if s["save"] == "bf16":
        return hidden, pre.to(s["x"].dtype)
    return hidden, _unpack8(*_pack8(pre)).to(s["x"].dtype)


def _plain_gated_backward(s):
    kept = _unpack8(*s["saved"]) if s["save"] == "8bit" else s["saved"].float()
    gate, up = kept.unbind(1)
    sig, dsig = _sigma(gate, s["act"])
    d = s["grad_hidden"].float()
    pre = torch.cat((d * up * (sig + gate * dsig), d * gate * sig), dim=1)
    grad_x, grad_weights = _plain_matmul_backward(s, pre, s["x"], s["weights"])
    hidden = gate * sig * up
    if s["offsets"] is not None:
        past = torch.arange(hidden.shape[0], device=hidden.device) >= s["offsets"][-1]
        hidden = hidden.masked_fill(past[:, None], 0.0)
    return grad_x, grad_weights, hidden.to(s["x"].dtype)


# -------------------------------------------------------------- one pass
def run(state):
    s = state
    op = s["op"]
    if not own:
        if op == "gated":
            return _plain_gated(s)
        if op == "gated_backward":
            return _plain_gated_backward(s)
        if op == "matmul":
            return _plain_matmul(s, s["x"], s["weights"]).to(s["x"].dtype)
        if op == "matmul_backward":
            return _plain_matmul_backward(s, s["grad_out"], s["x"], s["weights"])
        return _unpack8(*_pack8(s["x"])).to(s["x"].dtype)
    import latent_moe_output_gb300 as lt

    if op == "gated":
        saved = lt.Checkpoint8(*s["saved"]) if s["save"] == "8bit" else s["saved"]
        hidden = lt.expert_gated(s["x"], s["weights"], s["offsets"], activation=s["act"],
                                 hidden=s["hidden"], saved=saved)
        if s["save"] == "none":
            return hidden
        return hidden, lt.dequantize8(saved) if s["save"] == "8bit" else saved
    if op == "gated_backward":
        saved = lt.Checkpoint8(*s["saved"]) if s["save"] == "8bit" else s["saved"]
        return lt.expert_gated_backward(s["grad_hidden"], s["x"], s["weights"], saved,
                                        s["offsets"], activation=s["act"], grad_x=s["grad_x"],
                                        grad_weights=s["grad_weights"], hidden=s["hidden"],
                                        workspace=s["workspace"])
    if op == "matmul":
        return lt.expert_matmul(s["x"], s["weights"], s["offsets"], out=s["out"])
    if op == "matmul_backward":
        return lt.expert_matmul_backward(s["grad_out"], s["x"], s["weights"], s["offsets"],
                                         grad_x=s["grad_x"], grad_weights=s["grad_weights"])
    kept = lt.quantize8(s["x"], lt.Checkpoint8(s["values"], s["exponents"]))
    return lt.dequantize8(kept, out=s["out"])


# ------------------------------------------------------------------ work
def work(case):
    op, T, C = case["op"], case["T"], case["C"]
    if op == "checkpoint8":
        # The activations in, their 8 bits out and in again, the values out.
        packed = T * (C + -(-C // GROUP))
        return dict(bytes=4 * T * C + 2 * packed, flops=8 * T * C)
    K, E = case["K"], case["E"]
    n = T * K
    live = n * (1.0 - case["drop"])
    read = E * (1.0 - (1.0 - K * (1.0 - case["drop"]) / E) ** T) if E > 1 else 1.0
    if op in ("matmul", "matmul_backward"):
        M = case["M"]
        if op == "matmul":
            return dict(bytes=read * M * C * 2 + n * (C + M) * 2, flops=2 * live * M * C)
        return dict(bytes=(read + E) * M * C * 2 + n * (2 * C + M) * 2, flops=4 * live * M * C)
    F = case["F"]
    kept = {"none": 0, "bf16": 4 * F, "8bit": 2 * (F + -(-F // GROUP))}[case["save"]]
    if op == "gated":
        kept += 4 * F if case["save"] == "8bit" else 0  # returned as the values they stand for
        return dict(bytes=read * 2 * F * C * 2 + n * ((C + F) * 2 + kept), flops=4 * live * F * C)
    return dict(bytes=(read + E) * 2 * F * C * 2 + n * ((2 * C + 2 * F) * 2 + kept),
                flops=8 * live * F * C)


# --------------------------------------------------- definitions in 64 bits
def _exact_pack8(v):
    """The values that ``v`` [N, 2, F] or [N, C] (64 bits, finite) stands for after 8 bits."""
    out = v.clone()
    for a in range(0, v.shape[-1], GROUP):
        part = v[..., a:a + GROUP]
        top = part.abs().amax(-1, keepdim=True)
        unit = torch.exp2(torch.floor(torch.log2(top.clamp(min=1e-300))) - 6)
        unit = torch.where(torch.round(top / unit) > 127, 2 * unit, unit)
        out[..., a:a + GROUP] = torch.where(top > 0, torch.round(part / unit) * unit, part)
    return out


def _exact_act(g, act):
    if act == "silu":
        return g / (1 + torch.exp(-g))
    return 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))


def exact(case, seed):
    s = prepare(case, seed)
    op, x = s["op"], s["x"].double()
    if op == "checkpoint8":
        return _exact_pack8(x)
    w, n = s["weights"], x.shape[0]
    E, dev = w.shape[0], x.device
    bounds = [0, n] if s["offsets"] is None else s["offsets"].tolist()
    experts = [(e, slice(bounds[e], bounds[e + 1])) for e in range(E)
               if bounds[e] < bounds[e + 1]]
    zeros = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device=dev)  # noqa: E731
    if op in ("gated", "matmul"):
        out = zeros(n, w.shape[1])
        for e, part in experts:
            out[part] = x[part] @ w[e].double().t()
        if op == "matmul":
            return out
        gate, up = out.chunk(2, dim=1)
        hidden = _exact_act(gate, case["act"]) * up
        kept = out.unflatten(1, (2, -1))
        if s["save"] == "none":
            return hidden
        return hidden, kept if s["save"] == "bf16" else _exact_pack8(kept)
    hidden = None
    if op == "gated_backward":
        if s["save"] == "8bit":
            values, e8 = s["saved"]
            kept = values.double() * torch.exp2(
                e8.double() - 127).repeat_interleave(GROUP, dim=-1)[..., :values.shape[-1]]
        else:
            kept = s["saved"].double()
        kept.requires_grad_(True)
        hidden = _exact_act(kept[:, 0], case["act"]) * kept[:, 1]
        (grad,) = torch.autograd.grad(hidden, kept, s["grad_hidden"].double())
        grad = grad.flatten(1)
    else:
        grad = s["grad_out"].double()
    grad_x, grad_weights = zeros(*x.shape), zeros(*w.shape)
    for e, part in experts:
        grad_x[part] = grad[part] @ w[e].double()
        grad_weights[e] = grad[part].t() @ x[part]
    if op == "matmul_backward":
        return grad_x, grad_weights
    return grad_x, grad_weights, hidden.detach()
