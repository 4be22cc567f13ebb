"""Operators around the MoE layer: what each computes, in plain torch and by the library's entry points.

Four operators, as a pre-norm MoE block uses them:

* ``norm``      h = x + residual, y = h * rstd(h) * weight, and y once more as e4m3 codes with fp32 scales
                (one per 128 columns, or one per row) -- what FP8 expert GEMMs read.
* ``norm_bwd``  the gradient of that norm: dx (the gradient of x and of the residual alike) and dweight.
* ``balance``   per-expert counts, mean probabilities, the load-balance loss and the router z-loss of a batch of
                sequences with padding; ``route_step`` is the training step on them: the losses, and the gradient of
                both and of the routing weights with respect to the router's logits.
* ``combine_bwd`` the gradient of the weighted combine: of the expert rows, the routing weights, the shared expert's
                rows and its gate.

``own`` chooses between the two; both take what ``prepare`` made.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def _norm(name, T, H, residual=True, quant="none", weight="bf16"):
    return {"name": name, "op": "norm", "T": T, "H": H, "residual": residual, "quant": quant, "weight": weight}


def _norm_bwd(name, T, H, dh=True, weight="bf16"):
    return {"name": name, "op": "norm_bwd", "T": T, "H": H, "dh": dh, "weight": weight}


def _router(name, op, n_seq, L, E, K, mode=0, shared=False, padded=False):
    return {"name": name, "op": op, "n_seq": n_seq, "L": L, "E": E, "K": K, "mode": mode, "shared": shared,
            "padded": padded}


def _combine(name, T, K, H, E, shared=False):
    return {"name": name, "op": "combine_bwd", "T": T, "K": K, "H": H, "E": E, "shared": shared}


def listed():
    return [
        # one token of a decode step, ahead of the router: latency alone
        _norm("norm_T1_H2048", 1, 2048),
        # a decode batch whose experts read 8-bit rows; H is not a whole number of 128-column groups
        _norm("norm_q128_T32_H2880", 32, 2880, quant="group"),
        # a prefill chunk for 8-bit experts
        _norm("norm_q128_T4096_H2880", 4096, 2880, quant="group"),
        # one scale per row, the widest hidden size
        _norm("norm_qrow_T8191_H7168", 8191, 7168, quant="row", weight="f32"),
        # a short ragged micro-batch of a training step
        _norm_bwd("norm_bwd_T257_H2048", 257, 2048),
        # a full one
        _norm_bwd("norm_bwd_T8192_H7168", 8192, 7168, weight="f32"),
        # counts and losses of one prefill-sized batch (evaluation, monitoring)
        _router("balance_T2048_E128", "balance", 1, 2048, 128, 8),
        # eight padded sequences, logits with a shared-gate column: rows of 513 floats, no alignment
        _router("balance_T32768_E512", "balance", 8, 4096, 512, 10, shared=True, padded=True),
        # the router's training step on a small model
        _router("route_step_T100_E8", "route_step", 4, 25, 8, 2, padded=True),
        # sigmoid routing over many experts, a loss per sequence
        _router("route_step_T8192_E896", "route_step", 4, 2048, 896, 16, mode=1, padded=True),
        # the combine's gradient of a micro-batch
        _combine("combine_bwd_T509_K4_H2880", 509, 4, 2880, 32),
        # and of a large one with the gated shared expert
        _combine("combine_bwd_T8192_K10_H2048", 8192, 10, 2048, 512, shared=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(work(c)["bytes"] for c in listed())
    op = rng.choice(["norm", "norm_bwd", "balance", "route_step", "combine_bwd"])
    T = _log(rng, 1, 32768)
    H = 16 * _log(rng, 8, 512)
    E = _log(rng, 4, 1024)
    K = rng.randint(1, min(E, 20))
    if op == "norm":
        c = _norm("", T, H, rng.random() < 0.8, rng.choice(["none", "group", "row"]), rng.choice(["bf16", "f32"]))
    elif op == "norm_bwd":
        c = _norm_bwd("", T, H, rng.random() < 0.7, rng.choice(["bf16", "f32"]))
    elif op == "combine_bwd":
        c = _combine("", min(T, 16384), K, H, E, rng.random() < 0.5)
    else:
        n_seq = min(T, rng.choice([1, 1, 2, 3, 8, 32]))
        c = _router("", op, n_seq, max(1, T // n_seq), E, K, rng.randint(0, 1), rng.random() < 0.4, rng.random() < 0.6)
    del c["name"]
    size = "L" if "L" in c else "T"
    while work(c)["bytes"] > most:
        c[size] //= 2
    return c


# ------------------------------------------------------------------ inputs
def _groups(case):
    return {"none": 0, "group": -(-case["H"] // 128), "row": 1}[case["quant"]]


def _hidden(g, T, H, std=1.0):
    """Rows as a residual stream has them: a few columns far larger than the rest, rows of different size."""
    x = torch.randn(T, H, device="cuda", generator=g)
    x *= std * torch.exp(0.3 * torch.randn(T, 1, device="cuda", generator=g))
    x[:, torch.randint(0, H, (4,), device="cuda", generator=g)] *= 12.0
    return x.to(BF16)


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    op = case["op"]
    st = {"case": case}
    empty = lambda *shape, dtype=F32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    if op in ("norm", "norm_bwd"):
        T, H = case["T"], case["H"]
        w = 1.0 + 0.2 * torch.randn(H, device="cuda", generator=g)
        st["weight"] = w.to(BF16 if case["weight"] == "bf16" else F32)
        if op == "norm":
            st["x"] = _hidden(g, T, H, 0.5)
            st["residual"] = _hidden(g, T, H) if case["residual"] else None
            st["h"] = empty(T, H, dtype=BF16) if case["residual"] else None
            st["y"], st["rstd"] = empty(T, H, dtype=BF16), empty(T)
            if case["quant"] != "none":
                st["yq"] = empty(T, H, dtype=torch.float8_e4m3fn)
                st["yq_scale"] = empty(T, _groups(case))
        else:
            st["h"] = _hidden(g, T, H)
            st["rstd"] = torch.rsqrt(st["h"].float().square().mean(1) + EPS)
            st["dy"] = (torch.randn(T, H, device="cuda", generator=g) * 1e-2).to(BF16)
            st["dh"] = (torch.randn(T, H, device="cuda", generator=g) * 1e-2).to(BF16) if case["dh"] else None
            st["dx"], st["dweight"] = empty(T, H, dtype=BF16), empty(H)
    elif op in ("balance", "route_step"):
        S, L, E, K = case["n_seq"], case["L"], case["E"], case["K"]
        T, ld = S * L, E + (1 if case["shared"] else 0)
        st["logits"] = torch.randn(T, ld, device="cuda", generator=g) * 1.5
        st["logits"][:, : max(1, E // 16)] += 1.0  # some experts are hot
        if case["padded"]:
            n = torch.randint(0, L + 1, (S, 1), device="cuda", generator=g)
            n[S // 2] = L if S < 3 else 0  # one sequence is empty where there are several
            st["mask"] = (torch.arange(L, device="cuda")[None] < n).to(torch.uint8).reshape(T)
        else:
            st["mask"] = None
        # routing as the layer's forward pass gives it
        l = st["logits"][:, :E]
        key = l if case["mode"] == 0 else torch.sigmoid(l)
        v, ids = key.topk(K, dim=1)
        st["ids"] = ids.to(torch.int32)
        st["scale"] = 1.0 if case["mode"] == 0 else 2.5
        st["weights"] = torch.softmax(v, 1) if case["mode"] == 0 else 2.5 * v / v.sum(1, keepdim=True)
        st["counts"], st["mean_prob"] = empty(S, E, dtype=torch.int32), empty(S, E)
        st["valid"], st["losses"] = empty(S + 2, dtype=torch.int32), empty(2)
        if op == "route_step":
            st["grad_losses"] = torch.tensor([1e-2, 1e-3], device="cuda")
            st["d_weights"] = torch.randn(T, K, device="cuda", generator=g) * (1.0 / T)
            st["d_shared_gate"] = torch.randn(T, device="cuda", generator=g) * (1.0 / T) if case["shared"] else None
            st["dlogits"] = empty(T, ld)
    else:
        T, K, H, E = case["T"], case["K"], case["H"], case["E"]
        st["dout"] = (torch.randn(T, H, device="cuda", generator=g) * 1e-2).to(BF16)
        st["y"] = torch.randn(T * K, H, device="cuda", generator=g, dtype=BF16)
        # the order of a stable counting sort by expert
        ids = torch.rand(T, E, device="cuda", generator=g).topk(K, dim=1).indices.reshape(-1)
        order = torch.sort(ids, stable=True).indices
        f2r = torch.empty_like(order)
        f2r[order] = torch.arange(T * K, device="cuda")
        st["flat_to_row"] = f2r.to(torch.int32)
        st["weights"] = torch.softmax(torch.randn(T, K, device="cuda", generator=g), 1)
        st["dy"], st["d_weights"] = empty(T * K, H, dtype=BF16), empty(T, K)
        st["shared_y"] = st["shared_gate"] = st["d_shared_y"] = st["d_shared_gate"] = None
        if case["shared"]:
            st["shared_y"] = torch.randn(T, H, device="cuda", generator=g, dtype=BF16)
            st["shared_gate"] = torch.sigmoid(torch.randn(T, device="cuda", generator=g))
            st["d_shared_y"], st["d_shared_gate"] = empty(T, H, dtype=BF16), empty(T)
    return st


# ------------------------------------------------------------------ one pass
def run(st):
    op = st["case"]["op"]
    if own:
        return _OWN[op](st)
    return _PLAIN[op](st)


# ---- the library's entry points, into buffers that the caller keeps
def _scratch(st, nbytes):
    if "scratch" not in st:
        st["scratch"] = torch.zeros(max(nbytes(), 256), dtype=torch.uint8, device="cuda")
    return st["scratch"]


def _own_norm(st):
    from mixture_experts_layer_07_gb300 import ops
    q = st["case"]["quant"]
    ops.add_rmsnorm(st["x"], st["weight"], EPS, st["y"], residual=st["residual"], h=st["h"], rstd=st["rstd"],
                    yq=st.get("yq"), yq_scale=st.get("yq_scale"), q_group=128 if q == "group" else 0)
    return {k: st[k] for k in ("h", "y", "rstd", "yq", "yq_scale") if st.get(k) is not None}


def _own_norm_bwd(st):
    from mixture_experts_layer_07_gb300 import ops
    s = _scratch(st, lambda: ops.add_rmsnorm_backward_scratch_bytes(*st["h"].shape))
    ops.add_rmsnorm_backward(st["dy"], st["h"], st["rstd"], st["weight"], st["dx"], st["dweight"], s, dh=st["dh"])
    return {"dx": st["dx"], "dweight": st["dweight"]}


def _own_balance(st):
    from mixture_experts_layer_07_gb300 import ops
    c = st["case"]
    s = _scratch(st, lambda: ops.balance_loss_scratch_bytes(c["n_seq"] * c["L"], c["E"], c["n_seq"]))
    ops.balance_loss(st["logits"], st["ids"], c["E"], st["counts"], st["mean_prob"], st["valid"], st["losses"], s,
                     n_seq=c["n_seq"], mode=c["mode"], token_mask=st["mask"])
    return {k: st[k] for k in ("counts", "mean_prob", "valid", "losses")}


def _own_route_step(st):
    from mixture_experts_layer_07_gb300 import ops
    c = st["case"]
    out = _own_balance(st)
    ops.route_backward(st["logits"], st["ids"], c["E"], st["dlogits"], mode=c["mode"], scale=st["scale"],
                       weights=st["weights"], d_weights=st["d_weights"], d_shared_gate=st["d_shared_gate"],
                       token_mask=st["mask"], n_seq=c["n_seq"], counts=st["counts"], valid=st["valid"],
                       grad_losses=st["grad_losses"])
    return {**out, "dlogits": st["dlogits"]}


def _own_combine_bwd(st):
    from mixture_experts_layer_07_gb300 import ops
    c = st["case"]
    ops.unpermute_backward(st["dout"], st["flat_to_row"], st["weights"], c["T"], c["K"], c["H"], y=st["y"],
                           dy=st["dy"], d_weights=st["d_weights"], shared_y=st["shared_y"],
                           shared_gate=st["shared_gate"], d_shared_y=st["d_shared_y"],
                           d_shared_gate=st["d_shared_gate"])
    return {k: st[k] for k in ("dy", "d_weights", "d_shared_y", "d_shared_gate") if st[k] is not None}


_OWN = {"norm": _own_norm, "norm_bwd": _own_norm_bwd, "balance": _own_balance, "route_step": _own_route_step,
        "combine_bwd": _own_combine_bwd}


# ---- plain forms: 32 bits throughout, one rounding at the end
def _quantise(y, group):
    """e4m3 codes (as the values they stand for, before the scale) and scales of y's column groups."""
    T, H = y.shape
    n = -(-H // group)
    p = torch.zeros(T, n * group, device=y.device)
    p[:, :H] = y
    p = p.view(T, n, group)
    s = p.abs().amax(2) / E4M3_MAX
    q = torch.where(s[..., None] > 0, p / s[..., None], 0.0)
    return q.view(T, n * group)[:, :H].to(torch.float8_e4m3fn), s


def _plain_norm(st):
    c = st["case"]
    h = st["x"].float()
    out = {}
    if st["residual"] is not None:
        h = h + st["residual"].float()
        out["h"] = h.to(BF16)
    rstd = torch.rsqrt((h * h).mean(1) + EPS)
    y = h * rstd[:, None] * st["weight"].float()
    out["y"], out["rstd"] = y.to(BF16), rstd
    if c["quant"] != "none":
        out["yq"], out["yq_scale"] = _quantise(y, 128 if c["quant"] == "group" else c["H"])
    return out


def _plain_norm_bwd(st):
    n = st["h"].float() * st["rstd"][:, None]  # the normalised rows
    dy = st["dy"].float()
    gw = dy * st["weight"].float()
    dx = st["rstd"][:, None] * (gw - n * (gw * n).mean(1, keepdim=True))
    if st["dh"] is not None:
        dx = dx + st["dh"].float()
    return {"dx": dx.to(BF16), "dweight": (dy * n).sum(0)}


def _probabilities(l, mode):
    """Rows of probabilities, and (mode 1) one minus the sigmoid of each logit."""
    m = l.amax(1, keepdim=True)
    if mode == 0:
        e = torch.exp(l - m)
        return e / e.sum(1, keepdim=True), None
    # sigmoids over their sum, both times exp(max(0, -m)) so that rows of very negative logits keep their digits
    a = torch.exp(-l.abs())
    s = torch.where(l > 0, torch.exp((-m).clamp(min=0)), torch.exp(l + (-m).clamp(min=0))) / (1 + a)
    return s / s.sum(1, keepdim=True), torch.where(l > 0, a, torch.ones_like(a)) / (1 + a)


def _parts(st):
    c = st["case"]
    S, L, E, K = c["n_seq"], c["L"], c["E"], c["K"]
    l = st["logits"][:, :E]
    p, tail = _probabilities(l, c["mode"])
    m = l.amax(1, keepdim=True)
    lse = m[:, 0] + torch.log(torch.exp(l - m).sum(1))
    on = torch.ones(S * L, device=l.device) if st["mask"] is None else (st["mask"] != 0).float()
    hits = torch.zeros(S * L, E, device=l.device).scatter_(1, st["ids"].long(), 1.0) * on[:, None]
    counts = hits.view(S, L, E).sum(1)
    nv = on.view(S, L).sum(1)
    full = (nv > 0).sum()
    f = counts * (E / K) / nv.clamp(min=1)[:, None]
    mean_p = (p * on[:, None]).view(S, L, E).sum(1) / nv.clamp(min=1)[:, None]
    total = nv.sum()
    balance = (f * mean_p).sum() / full.clamp(min=1)
    z = (lse * lse * on).sum() / total.clamp(min=1)
    out = {"counts": counts.to(torch.int32), "mean_prob": mean_p,
           "valid": torch.cat([nv, total[None], full[None].float()]).to(torch.int32),
           "losses": torch.stack([balance, z])}
    return out, (l, p, tail, lse, on, f, nv, total, full)


def _plain_balance(st):
    return _parts(st)[0]


def _plain_route_step(st):
    c = st["case"]
    S, L, E = c["n_seq"], c["L"], c["E"]
    out, (l, p, tail, lse, on, f, nv, total, full) = _parts(st)
    g_bal, g_z = st["grad_losses"][0], st["grad_losses"][1]
    # the balance loss: counts are constants, so only the mean probabilities carry a gradient
    a = (g_bal * f / (nv.clamp(min=1)[:, None] * full.clamp(min=1))).repeat_interleave(L, 0)
    d = p * (a - (a * p).sum(1, keepdim=True))
    if tail is not None:
        d = d * tail
    # the z-loss
    d = d + torch.exp(l - lse[:, None]) * (2 * g_z * lse / total.clamp(min=1))[:, None]
    # the routing weights
    w, gw, ids = st["weights"], st["d_weights"], st["ids"].long()
    t = w * (gw - (w * gw).sum(1, keepdim=True) / st["scale"])
    if tail is not None:
        t = t * tail.gather(1, ids)
    d = d.scatter_add(1, ids, t) * on[:, None]
    if c["shared"]:
        s = 1 / (1 + torch.exp(-st["logits"][:, E]))
        d = torch.cat([d, (st["d_shared_gate"] * s * (1 - s) * on)[:, None]], 1)
    return {**out, "dlogits": d}


def _plain_combine_bwd(st):
    c = st["case"]
    T, K, H = c["T"], c["K"], c["H"]
    dout, rows, w = st["dout"].float(), st["flat_to_row"].long(), st["weights"]
    out = {"d_weights": (st["y"][rows].float().view(T, K, H) * dout[:, None]).sum(2)}
    dy = torch.empty_like(st["dy"])
    dy[rows] = (w[:, :, None] * dout[:, None]).to(BF16).view(T * K, H)
    out["dy"] = dy
    if c["shared"]:
        out["d_shared_y"] = (st["shared_gate"][:, None] * dout).to(BF16)
        out["d_shared_gate"] = (dout * st["shared_y"].float()).sum(1)
    return out


_PLAIN = {"norm": _plain_norm, "norm_bwd": _plain_norm_bwd, "balance": _plain_balance,
          "route_step": _plain_route_step, "combine_bwd": _plain_combine_bwd}


# ------------------------------------------------------------------ the floor
def work(case):
    """Each input read once and each output written once; the products and sums."""
    op = case["op"]
    if op == "norm":
        T, H = case["T"], case["H"]
        per = 2 + 2 + (4 if case["residual"] else 0) + (1 if case["quant"] != "none" else 0)
        return {"bytes": T * H * per + T * 4 * (1 + _groups(case)) + H * (2 if case["weight"] == "bf16" else 4),
                "flops": 6 * T * H}
    if op == "norm_bwd":
        T, H = case["T"], case["H"]
        return {"bytes": T * H * (6 + (2 if case["dh"] else 0)) + 4 * T + H * (6 if case["weight"] == "bf16" else 8),
                "flops": 10 * T * H}
    if op in ("balance", "route_step"):
        S, E, K = case["n_seq"], case["E"], case["K"]
        T, g = S * case["L"], 1 if case["shared"] else 0
        nbytes = 4 * T * E + 4 * T * K + (T if case["padded"] else 0) + 8 * S * E
        flops = 6 * T * E
        if op == "route_step":
            nbytes += 4 * T * (E + g) + 8 * T * K + 8 * T * g
            flops += 10 * T * E
        return {"bytes": nbytes, "flops": flops}
    T, K, H = case["T"], case["K"], case["H"]
    nbytes = 2 * T * H + 4 * T * K * H + 12 * T * K + ((4 * T * H + 8 * T) if case["shared"] else 0)
    return {"bytes": nbytes, "flops": 3 * T * K * H}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    st = prepare(case, seed)
    D = torch.float64
    op = case["op"]
    if op == "norm":
        h = st["x"].to(D)
        out = {}
        if st["residual"] is not None:
            h = h + st["residual"].to(D)
            out["h"] = h
        rms = (h.pow(2).sum(1) / case["H"] + EPS).sqrt()
        y = (h / rms[:, None]) * st["weight"].to(D)
        out["y"], out["rstd"] = y, 1 / rms
        if case["quant"] != "none":
            # what the codes stand for before their rounding to 8 bits
            blocks = y.split(128 if case["quant"] == "group" else case["H"], dim=1)
            scale = torch.stack([b.abs().amax(1) / E4M3_MAX for b in blocks], 1)
            out["yq"] = torch.cat([b / scale[:, i: i + 1] for i, b in enumerate(blocks)], 1)
            out["yq_scale"] = scale
        return out
    if op == "norm_bwd":
        # differentiates the norm itself; rstd is the one that the forward pass kept, which the inputs fix
        h = st["h"].to(D).requires_grad_()
        w = st["weight"].to(D).requires_grad_()
        y = h * (h.pow(2).mean(1, keepdim=True) + EPS).rsqrt() * w
        dx, dw = torch.autograd.grad(y, (h, w), st["dy"].to(D))
        if st["dh"] is not None:
            dx = dx + st["dh"].to(D)
        return {"dx": dx, "dweight": dw}
    if op in ("balance", "route_step"):
        S, L, E, K = case["n_seq"], case["L"], case["E"], case["K"]
        full = st["logits"].to(D).requires_grad_()
        l = full[:, :E]
        prob = torch.softmax(l if case["mode"] == 0 else torch.nn.functional.logsigmoid(l), 1)
        keep = torch.ones(S * L, dtype=torch.bool, device="cuda") if st["mask"] is None else st["mask"].bool()
        seq = torch.arange(S * L, device="cuda") // L
        nv = torch.bincount(seq[keep], minlength=S)
        flat = (seq[:, None] * E + st["ids"].long())[keep].reshape(-1)
        counts = torch.bincount(flat, minlength=S * E).view(S, E)
        some = nv > 0
        n1 = nv.clamp(min=1).to(D)[:, None]
        mean_p = torch.zeros(S, E, dtype=D, device="cuda").index_add(0, seq[keep], prob[keep]) / n1
        per_seq = E * (counts.to(D) / (K * n1) * mean_p).sum(1)
        balance = per_seq.sum() / max(1, int(some.sum()))
        z = torch.logsumexp(l[keep], 1).pow(2).sum() / max(1, int(nv.sum()))
        out = {"counts": None, "valid": None, "mean_prob": mean_p.detach(),
               "losses": torch.stack([balance, z]).detach()}
        if op == "route_step":
            picked = l.gather(1, st["ids"].long())
            if case["mode"] == 0:
                w = torch.softmax(picked, 1)
            else:
                w = torch.sigmoid(picked)
                w = st["scale"] * w / w.sum(1, keepdim=True)
            total = st["grad_losses"][0].to(D) * balance + st["grad_losses"][1].to(D) * z
            total = total + (w * st["d_weights"].to(D))[keep].sum()
            if case["shared"]:
                total = total + (torch.sigmoid(full[:, E]) * st["d_shared_gate"].to(D))[keep].sum()
            out["dlogits"], = torch.autograd.grad(total, full)
        return out
    T, K, H = case["T"], case["K"], case["H"]
    y = st["y"].to(D).requires_grad_()
    w = st["weights"].to(D).requires_grad_()
    comb = (y[st["flat_to_row"].long()].view(T, K, H) * w[:, :, None]).sum(1)
    leaves = [y, w]
    if case["shared"]:
        sy, sg = st["shared_y"].to(D).requires_grad_(), st["shared_gate"].to(D).requires_grad_()
        comb = comb + sg[:, None] * sy
        leaves += [sy, sg]
    grads = torch.autograd.grad(comb, leaves, st["dout"].to(D))
    return dict(zip(("dy", "d_weights", "d_shared_y", "d_shared_gate"), grads))
