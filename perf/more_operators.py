"""The experts' gradient and the 8-bit activations that it starts from, in plain torch and by the library's entry points.

Four operators, as the backward pass of a pre-norm MoE block uses them:

* ``pack``       rows of activations as e4m3 codes with an fp32 scale per row and 128 columns, to be kept for the
                 backward pass (half the memory of bf16).
* ``unpack``     those codes as bf16 rows again.
* ``norm_bwd``   the gradient of the RMS norm whose input h was kept as such codes.
* ``experts_bwd`` the gradient of sort by expert, SwiGLU experts and weighted return, from the tokens (bf16, or codes)
                 and the gradient of the layer's output: of the tokens, of the routing weights and of the experts'
                 three matrices.  Gate and up products are computed again, nothing of the forward pass but the routing
                 is kept.

``own`` chooses between the two; both take what ``prepare`` made.
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases
def _rows(name, op, T, H):
    return {"name": name, "op": op, "T": T, "H": H}


def _norm_bwd(name, T, H, dh=True, weight="bf16"):
    return {"name": name, "op": "norm_bwd", "T": T, "H": H, "dh": dh, "weight": weight}


def _experts(name, T, H, E, K, I, x="bf16", frozen=False):
    return {"name": name, "op": "experts_bwd", "T": T, "H": H, "E": E, "K": K, "I": I, "x": x, "frozen": frozen}


def listed():
    return [
        # one token's row: latency alone
        _rows("pack_T1_H2048", "pack", 1, 2048),
        # the residual stream of a full training micro-batch, an odd number of rows
        _rows("pack_T8191_H7168", "pack", 8191, 7168),
        # a short ragged micro-batch; H is not a whole number of 128-column groups
        _rows("unpack_T257_H2880", "unpack", 257, 2880),
        # a large one, for the gate's weight gradient
        _rows("unpack_T16384_H2048", "unpack", 16384, 2048),
        # the norm's gradient of a short micro-batch
        _norm_bwd("norm_bwd_T257_H2048", 257, 2048),
        # and of a full one at the widest hidden size
        _norm_bwd("norm_bwd_T8192_H7168", 8192, 7168, weight="f32"),
        # a small model, few rows per expert and not a whole tile of them
        _experts("experts_bwd_T100_E8_K2", 100, 256, 8, 2, 128),
        # few tokens on many experts: most experts have a row or two, some none
        _experts("experts_bwd_T64_E512_K10", 64, 2048, 512, 10, 512),
        # a micro-batch on many small experts: about a tile of rows each
        _experts("experts_bwd_T2048_E128_K8", 2048, 2048, 128, 8, 768),
        # few wide experts from 8-bit tokens, some experts hot
        _experts("experts_bwd_T4096_E32_K4_q8", 4096, 2880, 32, 4, 2880, x="q8"),
        # experts that do not learn (adapters, or the gate alone): tokens and routing weights only
        _experts("experts_bwd_T1023_E32_K4_frozen", 1023, 2880, 32, 4, 2880, x="q8", frozen=True),
        # a shared expert with its gate: one expert that takes every token
        _experts("experts_bwd_T4096_shared", 4096, 2048, 1, 1, 512),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6e12, w["flops"] / 1e15)


def draw(rng):
    op = rng.choice(["pack", "unpack", "norm_bwd", "experts_bwd", "experts_bwd", "experts_bwd"])
    H = 16 * _log(rng, 8, 512)
    if op in ("pack", "unpack"):
        c = _rows("", op, _log(rng, 1, 32768), H)
    elif op == "norm_bwd":
        c = _norm_bwd("", _log(rng, 1, 32768), H, rng.random() < 0.7, rng.choice(["bf16", "f32"]))
    else:
        E = _log(rng, 1, 256)
        c = _experts("", _log(rng, 8, 8192), H, E, rng.randint(1, min(E, 12)), 16 * _log(rng, 4, 192),
                     rng.choice(["bf16", "bf16", "q8"]), rng.random() < 0.3)
    del c["name"]
    most = max(_cost(x) for x in listed() if x["op"] == op)
    while _cost(c) > most:
        if op == "experts_bwd" and c["E"] * c["I"] > 64 * c["T"]:
            c["I"] = max(16, c["I"] // 32 * 16)
        else:
            c["T"] //= 2
    return c


# ------------------------------------------------------------------ inputs
def _hidden(g, T, H, std=1.0):
    """Rows as a residual stream has them: a few columns far larger than the rest, rows of different size."""
    x = torch.randn(T, H, device="cuda", generator=g)
    x *= std * torch.exp(0.3 * torch.randn(T, 1, device="cuda", generator=g))
    x[:, torch.randint(0, H, (4,), device="cuda", generator=g)] *= 12.0
    return x.to(BF16)


def _normed(g, T, H):
    """Rows as a norm gives them."""
    x = _hidden(g, T, H).float()
    return (x * torch.rsqrt(x.square().mean(1, keepdim=True) + EPS)).to(BF16)


def _codes(x):
    """The codes and scales of x that a forward pass kept."""
    T, H = x.shape
    n = -(-H // 128)
    p = torch.zeros(T, n * 128, device="cuda")
    p[:, :H] = x
    p = p.view(T, n, 128)
    s = p.abs().amax(2) / E4M3_MAX
    q = torch.where(s[..., None] > 0, p / s[..., None], 0.0).clamp(-E4M3_MAX, E4M3_MAX)
    return q.view(T, n * 128)[:, :H].to(torch.float8_e4m3fn).contiguous(), s


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    op, T, H = case["op"], case["T"], case["H"]
    st = {"case": case}
    empty = lambda *shape, dtype=F32: torch.empty(*shape, dtype=dtype, device="cuda")  # noqa: E731
    rand = lambda *shape: torch.randn(*shape, device="cuda", generator=g)  # noqa: E731
    if op == "pack":
        st["x"] = _hidden(g, T, H)
        st["xq"], st["xq_scale"] = empty(T, H, dtype=torch.float8_e4m3fn), empty(T, -(-H // 128))
    elif op == "unpack":
        st["xq"], st["xq_scale"] = _codes(_hidden(g, T, H))
        st["x"] = empty(T, H, dtype=BF16)
    elif op == "norm_bwd":
        h = _hidden(g, T, H)
        st["rstd"] = torch.rsqrt(h.float().square().mean(1) + EPS)
        st["hq"], st["hq_scale"] = _codes(h)
        st["weight"] = (1.0 + 0.2 * rand(H)).to(BF16 if case["weight"] == "bf16" else F32)
        st["dy"] = (rand(T, H) * 1e-2).to(BF16)
        st["dh"] = (rand(T, H) * 1e-2).to(BF16) if case["dh"] else None
        st["dx"], st["dweight"] = empty(T, H, dtype=BF16), empty(H)
    else:
        E, K, I = case["E"], case["K"], case["I"]
        x = _normed(g, T, H)
        st["x"] = x if case["x"] == "bf16" else None
        st["xq"], st["xq_scale"] = _codes(x) if case["x"] == "q8" else (None, None)
        st["dout"] = (rand(T, H) * 1e-2).to(BF16)
        st["dx_add"] = (rand(T, H) * 1e-2).to(BF16)  # what reaches the tokens through the gate
        for name, shape, fan in (("w1", (E, I, H), H), ("w3", (E, I, H), H), ("w2", (E, H, I), I)):
            st[name] = (rand(*shape) * fan ** -0.5).to(BF16)
        # the routing that the forward pass kept: some experts are hot; rows in the order of a stable sort by expert
        logits = rand(T, E)
        logits[:, : max(1, E // 16)] += 1.0
        v, ids = logits.topk(K, dim=1)
        st["weights"] = torch.softmax(v, 1) if E > 1 else torch.sigmoid(v)
        order = torch.sort(ids.reshape(-1), stable=True).indices
        f2r = torch.empty_like(order)
        f2r[order] = torch.arange(T * K, device="cuda")
        st["row_to_flat"], st["flat_to_row"] = order.to(torch.int32), f2r.to(torch.int32)
        off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
        off[1:] = torch.bincount(ids.reshape(-1), minlength=E).cumsum(0)
        st["offsets"] = off
        st["dx"], st["d_weights"] = empty(T, H, dtype=BF16), empty(T, K)
        for name in ("w1", "w3", "w2"):
            st["d" + name] = None if case["frozen"] else torch.empty_like(st[name])
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
        st["scratch"] = torch.empty(max(nbytes(), 256), dtype=torch.uint8, device="cuda")
    return st["scratch"]


def _own_pack(st):
    from mixture_experts_layer_07_gb300 import ops
    ops.pack_q8(st["x"], st["xq"], st["xq_scale"])
    return {"xq": st["xq"], "xq_scale": st["xq_scale"]}


def _own_unpack(st):
    from mixture_experts_layer_07_gb300 import ops
    ops.unpack_q8(st["xq"], st["xq_scale"], st["x"])
    return {"x": st["x"]}


def _own_norm_bwd(st):
    from mixture_experts_layer_07_gb300 import ops
    s = _scratch(st, lambda: ops.add_rmsnorm_backward_scratch_bytes(*st["dy"].shape))
    ops.add_rmsnorm_backward_q8(st["dy"], st["hq"], st["hq_scale"], st["rstd"], st["weight"], st["dx"],
                                st["dweight"], s, dh=st["dh"])
    return {"dx": st["dx"], "dweight": st["dweight"]}


def _own_experts_bwd(st):
    from mixture_experts_layer_07_gb300 import ops
    c = st["case"]
    s = _scratch(st, lambda: ops.experts_backward_scratch_bytes(c["T"], c["H"], c["E"], c["K"], c["I"]))
    ops.experts_backward(st["dout"], st["offsets"], st["row_to_flat"], st["flat_to_row"], st["weights"], st["w1"],
                         st["w3"], st["w2"], s, x=st["x"], xq=st["xq"], xq_scale=st["xq_scale"],
                         dx_add=st["dx_add"], dx=st["dx"], d_weights=st["d_weights"], dw1=st["dw1"],
                         dw3=st["dw3"], dw2=st["dw2"])
    return {k: st[k] for k in ("dx", "d_weights", "dw1", "dw3", "dw2") if st[k] is not None}


_OWN = {"pack": _own_pack, "unpack": _own_unpack, "norm_bwd": _own_norm_bwd, "experts_bwd": _own_experts_bwd}


# ---- plain forms: 32 bits throughout, one rounding at the end
def _plain_pack(st):
    T, H = st["x"].shape
    n = -(-H // 128)
    p = torch.zeros(T, n * 128, device="cuda")
    p[:, :H] = st["x"]
    p = p.view(T, n, 128)
    s = p.abs().amax(2) / E4M3_MAX
    q = torch.where(s[..., None] > 0, p / s[..., None], 0.0)
    return {"xq": q.view(T, n * 128)[:, :H].to(torch.float8_e4m3fn), "xq_scale": s}


def _decoded(q, s):
    return q.float() * s.repeat_interleave(128, 1)[:, : q.shape[1]]


def _plain_unpack(st):
    return {"x": _decoded(st["xq"], st["xq_scale"]).to(BF16)}


def _plain_norm_bwd(st):
    n = _decoded(st["hq"], st["hq_scale"]) * st["rstd"][:, None]  # the normalised rows
    dy = st["dy"].float()
    gw = dy * st["weight"].float()
    dx = st["rstd"][:, None] * (gw - n * (gw * n).mean(1, keepdim=True))
    if st["dh"] is not None:
        dx = dx + st["dh"].float()
    return {"dx": dx.to(BF16), "dweight": (dy * n).sum(0)}


def _tokens(st):
    """The tokens' rows that the products take: bf16, or the codes rounded to bf16."""
    return st["x"] if st["x"] is not None else _decoded(st["xq"], st["xq_scale"]).to(BF16)


def _plain_experts_bwd(st):
    c = st["case"]
    T, H, E, K = c["T"], c["H"], c["E"], c["K"]
    r2f, f2r, off = st["row_to_flat"].long(), st["flat_to_row"].long(), st["offsets"].long()
    # the experts' rows, each expert's padded with zeros to those of the fullest
    M = int((off[1:] - off[:-1]).max())
    row = torch.arange(T * K, device="cuda")
    e = torch.searchsorted(off, row, right=True) - 1
    at = e * M + row - off[e]

    def padded(rows):
        p = torch.zeros(E * M, rows.shape[1], device="cuda")
        p[at] = rows.float()
        return p.view(E, M, -1)

    x, dout = padded(_tokens(st)[r2f // K]), padded(st["dout"][r2f // K])
    w = padded(st["weights"].reshape(-1)[r2f][:, None])
    w1, w3, w2 = st["w1"].float(), st["w3"].float(), st["w2"].float()
    g, u, a = x @ w1.transpose(1, 2), x @ w3.transpose(1, 2), dout @ w2
    s = 1 / (1 + torch.exp(-g))
    act = g * s * u
    dw = (a * act).sum(2).view(-1)[at]
    a = w * a
    dg, du = a * u * s * (1 + g * (1 - s)), a * g * s
    dxp = (dg @ w1 + du @ w3).view(E * M, H)[at]
    out = {"d_weights": dw[f2r].view(T, K),
           "dx": (dxp[f2r].view(T, K, H).sum(1) + st["dx_add"].float()).to(BF16)}
    if not c["frozen"]:
        out["dw1"] = (dg.transpose(1, 2) @ x).to(BF16)
        out["dw3"] = (du.transpose(1, 2) @ x).to(BF16)
        out["dw2"] = (dout.transpose(1, 2) @ (w * act)).to(BF16)
    return out


_PLAIN = {"pack": _plain_pack, "unpack": _plain_unpack, "norm_bwd": _plain_norm_bwd,
          "experts_bwd": _plain_experts_bwd}


# ------------------------------------------------------------------ the floor
def work(case):
    """Each input read once and each output written once; the products and sums."""
    op, T, H = case["op"], case["T"], case["H"]
    scales = 4 * T * -(-H // 128)
    if op in ("pack", "unpack"):
        return {"bytes": 3 * T * H + scales, "flops": 2 * T * H}
    if op == "norm_bwd":
        return {"bytes": T * H * (5 + (2 if case["dh"] else 0)) + scales + 4 * T
                + H * (6 if case["weight"] == "bf16" else 8), "flops": 11 * T * H}
    E, K, I = case["E"], case["K"], case["I"]
    R = T * K
    tokens = T * H * (2 if case["x"] == "bf16" else 1) + (scales if case["x"] == "q8" else 0)
    # experts without a row are not read, but their gradients are written (as zeros)
    nbytes = tokens + 6 * T * H + 16 * R + 6 * min(E, R) * H * I + (0 if case["frozen"] else 6 * E * H * I)
    return {"bytes": nbytes, "flops": (10 if case["frozen"] else 16) * R * H * I}


# ------------------------------------------------------------------ the definitions in 64 bits
def _decoded64(q, s):
    return q.float().double() * s.double().repeat_interleave(128, 1)[:, : q.shape[1]]


def exact(case, seed):
    st = prepare(case, seed)
    D = torch.float64
    op = case["op"]
    if op == "pack":
        # what the codes stand for before their rounding to 8 bits
        blocks = st["x"].to(D).split(128, dim=1)
        scale = torch.stack([b.abs().amax(1) / E4M3_MAX for b in blocks], 1)
        return {"xq": torch.cat([b / scale[:, i: i + 1] for i, b in enumerate(blocks)], 1), "xq_scale": scale}
    if op == "unpack":
        return {"x": _decoded64(st["xq"], st["xq_scale"])}
    if op == "norm_bwd":
        # y = h rstd(h) weight with rstd as the forward pass kept it: d rstd = -rstd^3 <h, dh> / H
        h, r = _decoded64(st["hq"], st["hq_scale"]), st["rstd"].to(D)[:, None]
        dy, w = st["dy"].to(D), st["weight"].to(D)
        dx = dy * w * r - h * r ** 3 * (dy * w * h).sum(1, keepdim=True) / case["H"]
        if st["dh"] is not None:
            dx = dx + st["dh"].to(D)
        return {"dx": dx, "dweight": (dy * h * r).sum(0)}
    T, K, E = case["T"], case["K"], case["E"]
    x = st["x"] if st["x"] is not None else _decoded64(st["xq"], st["xq_scale"]).to(BF16)
    x = x.to(D).requires_grad_()
    wt = st["weights"].to(D).requires_grad_()
    ids = torch.empty(T * K, dtype=torch.long, device="cuda")
    off = st["offsets"].tolist()
    for e in range(E):
        ids[st["row_to_flat"][off[e]: off[e + 1]].long()] = e
    dx, dwt = st["dx_add"].to(D), torch.zeros_like(wt)
    grads = {n: None if case["frozen"] else torch.zeros_like(st[n], dtype=F32) for n in ("w1", "w3", "w2")}
    # expert by expert, by differentiation of what the forward pass computes
    for e in range(E):
        flat = (ids == e).nonzero()[:, 0]
        if not len(flat):
            continue
        leaves = [st[n][e].to(D).requires_grad_(not case["frozen"]) for n in ("w1", "w3", "w2")]
        tok = flat // K
        xe, we = x.detach()[tok].requires_grad_(), wt.detach().view(-1)[flat].requires_grad_()
        gate = xe @ leaves[0].t()
        y = (gate * torch.sigmoid(gate) * (xe @ leaves[1].t())) @ leaves[2].t()
        wanted = [xe, we] + ([] if case["frozen"] else leaves)
        got = torch.autograd.grad(y * we[:, None], wanted, st["dout"][tok].to(D))
        dx = dx.index_add(0, tok, got[0])
        dwt.view(-1)[flat] = got[1]
        for n, v in zip(("w1", "w3", "w2"), got[2:]):
            grads[n][e] = v.float()
    out = {"dx": dx, "d_weights": dwt.detach()}
    if not case["frozen"]:
        out |= {"d" + n: v for n, v in grads.items()}
    return out
