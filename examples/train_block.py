"""A training step of a pre-norm MoE block on the library's operators.

    h      = x + residual                    moe_add_rmsnorm
    y      = rmsnorm(h) * norm_weight
    logits = y . wg^T                        moe_router_gemm
    ids, w = top-K routing                   moe_topk_route
    e      = experts(permute(y))             moe_permute, moe_grouped_gemm
    out    = h + combine(e, w)               moe_unpermute
    loss   = mean (out - target)^2 / 2 + alpha * balance + beta * z      moe_balance_loss

and back: moe_experts_backward gives the gradients of y (through the experts), of
the routing weights and of the experts' matrices from y, the routing and d_out
alone, moe_route_backward those of the logits (with both losses),
moe_add_rmsnorm_backward those of x and of the norm's weight.  Only the gate's
two small products backwards are torch.  Gate, norm, experts (fp32 copies of
their bf16 weights) and x learn.

With q8 the backward pass reads the two activations that it needs, h and y, as
e4m3 codes (moe_pack_q8, and what the norm writes): half the memory per layer in
a model that keeps only those.  This one block has its bf16 buffers besides.
The forward pass feeds the experts y in bf16, so the gradients are those at the
values that the codes stand for.

    python examples/train_block.py [steps] [q8]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from mixture_experts_layer_07_gb300 import ops  # noqa: E402

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
EPS = 1e-6


class Block:
    """Weights and buffers of one block for batches of n_seq x L tokens."""

    def __init__(self, n_seq=8, L=64, H=256, E=16, K=2, I=128, seed=0, alpha=1e-2, beta=1e-3,
                 q8=False):
        g = torch.Generator("cuda").manual_seed(seed)
        rand = lambda *s, std=1.0: torch.randn(*s, device="cuda", generator=g) * std  # noqa: E731
        self.n_seq, self.T, self.H, self.E, self.K, self.I = n_seq, n_seq * L, H, E, K, I
        T, R = self.T, self.T * K
        self.wg = rand(E, H, std=H ** -0.5)
        self.norm = torch.ones(H, device="cuda")
        self.w1, self.w3 = (rand(E, I, H, std=H ** -0.5).to(BF16) for _ in range(2))
        self.w2 = rand(E, H, I, std=I ** -0.5).to(BF16)
        self.grad_losses = torch.tensor([alpha, beta], device="cuda")
        e = lambda *s, dtype=F32: torch.empty(*s, dtype=dtype, device="cuda")  # noqa: E731
        self.h, self.y, self.moe = (e(T, H, dtype=BF16) for _ in range(3))
        self.q8 = q8
        if q8:
            codes = lambda: (e(T, H, dtype=torch.float8_e4m3fn), e(T, -(-H // 128)))  # noqa: E731
            (self.hq, self.hs), (self.yq, self.ys) = codes(), codes()
        self.rstd, self.logits, self.weights = e(T), e(T, E), e(T, K)
        self.ids, self.offsets = e(T, K, dtype=I32), e(E + 1, dtype=I32)
        self.r2f, self.f2r = e(R, dtype=I32), e(R, dtype=I32)
        self.xp, self.rows = (e(R, H, dtype=BF16) for _ in range(2))
        self.hact = e(R, I, dtype=BF16)
        self.counts, self.mean_prob = e(n_seq, E, dtype=I32), e(n_seq, E)
        self.valid, self.losses = e(n_seq + 2, dtype=I32), e(2)
        self.d_weights, self.d_logits = e(T, K), e(T, E)
        self.dy, self.dx, self.d_norm = e(T, H, dtype=BF16), e(T, H, dtype=BF16), e(H)
        self.experts = [w.float() for w in (self.w1, self.w3, self.w2)]
        self.d_experts = [torch.empty_like(w) for w in self.experts]
        zeros = lambda n: torch.zeros(max(n, 256), dtype=torch.uint8, device="cuda")  # noqa: E731
        self.s_permute = zeros(ops.permute_scratch_bytes(T, E, K))
        self.s_gemm = zeros(ops.grouped_gemm_scratch_bytes(R, E))
        self.s_balance = zeros(ops.balance_loss_scratch_bytes(T, E, n_seq))
        self.s_experts = zeros(ops.experts_backward_scratch_bytes(T, H, E, K, I))
        self.s_norm = zeros(ops.add_rmsnorm_backward_scratch_bytes(T, H))
        self.status = torch.zeros(1, dtype=I32, device="cuda")

    def forward(self, x, residual, mask):
        T, H, E, K = self.T, self.H, self.E, self.K
        q = dict(yq=self.yq, yq_scale=self.ys) if self.q8 else {}
        ops.add_rmsnorm(x, self.norm, EPS, self.y, residual=residual, h=self.h, rstd=self.rstd, **q)
        if self.q8:
            ops.pack_q8(self.h, self.hq, self.hs)
        ops.router_gemm(self.y, self.wg, None, self.logits)
        ops.topk_route(self.logits, E, K, ops.MODE_SOFTMAX, 1.0, self.ids, self.weights)
        ops.permute(self.y, self.ids, E, self.offsets, self.r2f, self.f2r, self.xp, self.s_permute,
                    self.status)
        ops.grouped_gemm(self.xp, self.offsets, E, H, self.I, self.w1, self.w3, self.w2, self.hact,
                         self.rows, self.s_gemm, dev_status=self.status)
        ops.unpermute(self.rows, self.f2r, self.weights, T, K, H, self.moe)
        ops.balance_loss(self.logits, self.ids, E, self.counts, self.mean_prob, self.valid,
                         self.losses, self.s_balance, n_seq=self.n_seq, token_mask=mask,
                         dev_status=self.status)
        return self.h.float() + self.moe.float()

    def backward(self, d_out, mask):
        """Gradients of x (and the residual), the gate and the norm's weight; the experts' are
        left in d_experts."""
        d_out = d_out.to(BF16)
        y = dict(xq=self.yq, xq_scale=self.ys) if self.q8 else dict(x=self.y)
        dw1, dw3, dw2 = self.d_experts
        ops.experts_backward(d_out, self.offsets, self.r2f, self.f2r, self.weights, self.w1, self.w3,
                             self.w2, self.s_experts, **y, dx=self.dy, d_weights=self.d_weights,
                             dw1=dw1, dw3=dw3, dw2=dw2, dev_status=self.status)
        ops.route_backward(self.logits, self.ids, self.E, self.d_logits, weights=self.weights,
                           d_weights=self.d_weights, token_mask=mask, n_seq=self.n_seq,
                           counts=self.counts, valid=self.valid, grad_losses=self.grad_losses,
                           dev_status=self.status)
        if self.q8:
            ops.unpack_q8(self.yq, self.ys, self.y)  # y's memory could have been another's in between
        d_gate = self.d_logits.t() @ self.y.float()
        # the experts' part comes back rounded to bf16, and the sum is rounded once more
        dy = (self.d_logits @ self.wg + self.dy.float()).to(BF16)
        if self.q8:
            ops.add_rmsnorm_backward_q8(dy, self.hq, self.hs, self.rstd, self.norm, self.dx,
                                        self.d_norm, self.s_norm, dh=d_out)
        else:
            ops.add_rmsnorm_backward(dy, self.h, self.rstd, self.norm, self.dx, self.d_norm,
                                     self.s_norm, dh=d_out)
        return self.dx, d_gate, self.d_norm

    def update(self, d_gate, d_norm, lr):
        self.wg -= lr * d_gate
        self.norm -= lr * d_norm
        for w, master, d in zip((self.w1, self.w3, self.w2), self.experts, self.d_experts):
            master -= lr * d
            w.copy_(master)


def train(steps=40, lr=0.5, **kw):
    """Loss, balance and z-loss of each step on one batch of random data."""
    b = Block(**kw)
    g = torch.Generator("cuda").manual_seed(1)
    T, H = b.T, b.H
    x = (torch.randn(T, H, device="cuda", generator=g) + 0.5).to(BF16)  # skewed: some experts hot
    residual = torch.randn(T, H, device="cuda", generator=g).to(BF16)
    target = torch.randn(T, H, device="cuda", generator=g)
    L = T // b.n_seq
    n = torch.randint(L // 2, L + 1, (b.n_seq, 1), device="cuda", generator=g)
    mask = (torch.arange(L, device="cuda")[None] < n).reshape(T)
    scale = mask[:, None].float() / (mask.sum() * H)
    history = []
    for _ in range(steps):
        out = b.forward(x, residual, mask)
        diff = out - target
        task = 0.5 * (diff.square() * scale).sum()
        dx, d_gate, d_norm = b.backward(diff * scale, mask)
        history.append((float(task), *b.losses.tolist()))
        b.update(d_gate, d_norm, lr)
        x = (x.float() - lr * T * H * 0.02 * dx.float()).to(BF16)
    if int(b.status.item()):
        raise RuntimeError(f"device status {int(b.status.item())}")
    return b, history


if __name__ == "__main__":
    block, hist = train(int(sys.argv[1]) if len(sys.argv) > 1 else 40, q8="q8" in sys.argv[2:])
    for i in sorted({0, len(hist) // 4, len(hist) // 2, len(hist) - 1}):
        print("step %3d   task %.4f   balance %.4f   z %.4f" % (i, *hist[i]))
    print("tokens per expert:", block.counts.sum(0).tolist())
