"""A training step of a pre-norm MoE block on the library's operators.

    h      = x + residual                    moe_add_rmsnorm
    y      = rmsnorm(h) * norm_weight
    logits = y . wg^T                        moe_router_gemm
    ids, w = top-K routing                   moe_topk_route
    e      = experts(permute(y))             moe_permute, moe_grouped_gemm
    out    = h + combine(e, w)               moe_unpermute
    loss   = mean (out - target)^2 / 2 + alpha * balance + beta * z      moe_balance_loss

and back: moe_unpermute_backward gives the gradients of the expert rows and of
the routing weights, moe_route_backward those of the logits (with both losses),
moe_add_rmsnorm_backward those of x and of the norm's weight.  What the library
has no kernel for -- the experts' and the gate's own matrix products backwards
-- is torch here.  The experts are kept; the gate, the norm's weight and x learn.

    python examples/train_block.py [steps]
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

    def __init__(self, n_seq=8, L=64, H=256, E=16, K=2, I=128, seed=0, alpha=1e-2, beta=1e-3):
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
        self.rstd, self.logits, self.weights = e(T), e(T, E), e(T, K)
        self.ids, self.offsets = e(T, K, dtype=I32), e(E + 1, dtype=I32)
        self.r2f, self.f2r = e(R, dtype=I32), e(R, dtype=I32)
        self.xp, self.rows, self.d_rows = (e(R, H, dtype=BF16) for _ in range(3))
        self.hact = e(R, I, dtype=BF16)
        self.counts, self.mean_prob = e(n_seq, E, dtype=I32), e(n_seq, E)
        self.valid, self.losses = e(n_seq + 2, dtype=I32), e(2)
        self.d_weights, self.d_logits = e(T, K), e(T, E)
        self.dx, self.d_norm = e(T, H, dtype=BF16), e(H)
        zeros = lambda n: torch.zeros(max(n, 256), dtype=torch.uint8, device="cuda")  # noqa: E731
        self.s_permute = zeros(ops.permute_scratch_bytes(T, E, K))
        self.s_gemm = zeros(ops.grouped_gemm_scratch_bytes(R, E))
        self.s_balance = zeros(ops.balance_loss_scratch_bytes(T, E, n_seq))
        self.s_norm = zeros(ops.add_rmsnorm_backward_scratch_bytes(T, H))
        self.status = torch.zeros(1, dtype=I32, device="cuda")

    def forward(self, x, residual, mask):
        T, H, E, K = self.T, self.H, self.E, self.K
        ops.add_rmsnorm(x, self.norm, EPS, self.y, residual=residual, h=self.h, rstd=self.rstd)
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
        """Gradients of x (and the residual), the gate and the norm's weight."""
        T, H, E, K = self.T, self.H, self.E, self.K
        d_out = d_out.to(BF16)
        ops.unpermute_backward(d_out, self.f2r, self.weights, T, K, H, y=self.rows, dy=self.d_rows,
                               d_weights=self.d_weights)
        ops.route_backward(self.logits, self.ids, E, self.d_logits, weights=self.weights,
                           d_weights=self.d_weights, token_mask=mask, n_seq=self.n_seq,
                           counts=self.counts, valid=self.valid, grad_losses=self.grad_losses,
                           dev_status=self.status)
        d_gate = self.d_logits.t() @ self.y.float()
        dy = self.d_logits @ self.wg + self._experts_backward()
        ops.add_rmsnorm_backward(dy.to(BF16), self.h, self.rstd, self.norm, self.dx, self.d_norm,
                                 self.s_norm, dh=d_out)
        return self.dx, d_gate, self.d_norm

    def _experts_backward(self):
        """The gradient that reaches y through the experts' products (torch)."""
        d_xp = torch.empty_like(self.xp, dtype=F32)
        off = self.offsets.tolist()
        for e in range(self.E):
            a, b = off[e], off[e + 1]
            x, w1, w3, w2 = (t.float() for t in (self.xp[a:b], self.w1[e], self.w3[e], self.w2[e]))
            g, u = x @ w1.t(), x @ w3.t()
            d_act = self.d_rows[a:b].float() @ w2
            s = torch.sigmoid(g)
            d_xp[a:b] = (d_act * u * s * (1 + g * (1 - s))) @ w1 + (d_act * g * s) @ w3
        return d_xp[self.f2r.long()].view(self.T, self.K, self.H).sum(1)


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
        b.wg -= lr * d_gate
        b.norm -= lr * d_norm
        x = (x.float() - lr * T * H * 0.02 * dx.float()).to(BF16)
    if int(b.status.item()):
        raise RuntimeError(f"device status {int(b.status.item())}")
    return b, history


if __name__ == "__main__":
    block, hist = train(int(sys.argv[1]) if len(sys.argv) > 1 else 40)
    for i in sorted({0, len(hist) // 4, len(hist) // 2, len(hist) - 1}):
        print("step %3d   task %.4f   balance %.4f   z %.4f" % (i, *hist[i]))
    print("tokens per expert:", block.counts.sum(0).tolist())
