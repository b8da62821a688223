"""A residual MLP block in microscaled precision: one forward pass for serving and one
training step, on the library's entry points.

    x, r  --gge_rmsnorm-->  h = x + r,  codes of norm(h)
    codes, W1  --gge_gemm_mx-->  u,  a = silu(u)
    a  --gge_mx_quantize-->  codes  --gge_gemm_mx (W2)-->  y

Backward: the gradients' products contract over the other dimension, so their operands
are quantised along it -- transposed views, and W2 once more along its other side:

    da = dy W2, du = silu'(u) da  (one product, gge_gemm_mx_dact)      dW2 = dy^T a
    dn = du W1                                                       dW1 = du^T n
    dn, h  --gge_rmsnorm_bwd-->  the gradient of x and r, and of the norm's weight

    python examples/low_precision_mlp.py [tokens] [width] [hidden] [format]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from grouped_gemm_epilogues_gb300 import binding as gge  # noqa: E402

EPS = 1e-5


def quantised(x, fmt):
    """x (rows, cols; a transposed view is fine) as a microscaled matrix."""
    t = None
    if fmt == "nvfp4":   # a program would keep this scale from calibration
        t = (x.abs().max().float() / 2688.0).clamp_min(1e-20).reshape(1)
    q = gge.mx_empty(x.shape[0], x.shape[1], fmt, device=x.device, tensor_scale=t)
    gge.gge_mx_quantize(x, q)
    return q


class Block:
    """Weights as a program keeps them: bf16 masters and their codes, laid out once."""

    def __init__(self, width, hidden, fmt, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def draw(n, k):
            return (torch.randn(n, k, generator=g, device=device) / k ** 0.5).bfloat16()

        self.fmt, self.width, self.hidden = fmt, width, hidden
        self.norm = torch.ones(width, dtype=torch.bfloat16, device=device)
        self.w1, self.w2 = draw(hidden, width), draw(width, hidden)
        self.refresh()

    def refresh(self):
        """The codes of the weights, after an update."""
        self.q1, self.q2 = quantised(self.w1, self.fmt), quantised(self.w2, self.fmt)
        self.q1t, self.q2t = quantised(self.w1.t(), self.fmt), quantised(self.w2.t(), self.fmt)

    def forward(self, x, r, keep=False):
        tokens, dev = x.shape[0], x.device
        h = torch.empty_like(x)
        inv = torch.empty(tokens, device=dev)
        n = torch.empty_like(x)
        if self.fmt == "nvfp4":   # the tensor scale is taken of the norm's output
            gge.gge_rmsnorm(x, self.norm, Y=n, residual=r, residual_out=h, inv_rms=inv, eps=EPS)
            qn = quantised(n, self.fmt)
        else:
            qn = gge.mx_empty(tokens, self.width, self.fmt, device=dev)
            gge.gge_rmsnorm(x, self.norm, Y=n if keep else None, residual=r, residual_out=h, Q=qn,
                            inv_rms=inv, eps=EPS)
        u = torch.empty(tokens, self.hidden, dtype=x.dtype, device=dev)
        a = torch.empty_like(u)
        gge.gge_gemm_mx(qn, self.q1, D=u, PostAct=a, act="silu")
        y = torch.empty_like(x)
        gge.gge_gemm_mx(quantised(a, self.fmt), self.q2, D=y)
        return y, h, (h, inv, n, u, a) if keep else None

    def backward(self, dy, dh, saved):
        h, inv, n, u, a = saved
        dev, dt = dy.device, dy.dtype
        du = torch.empty_like(u)
        gge.gge_gemm_mx_dact(quantised(dy, self.fmt), self.q2t, u, du, "silu")
        dn = torch.empty_like(n)
        gge.gge_gemm_mx(quantised(du, self.fmt), self.q1t, D=dn)
        dw2 = torch.empty(self.width, self.hidden, device=dev)
        gge.gge_gemm_mx(quantised(dy.t(), self.fmt), quantised(a.t(), self.fmt), D=dw2)
        dw1 = torch.empty(self.hidden, self.width, device=dev)
        gge.gge_gemm_mx(quantised(du.t(), self.fmt), quantised(n.t(), self.fmt), D=dw1)
        dx = torch.empty(dy.shape, dtype=dt, device=dev)
        dnorm = torch.empty(self.width, device=dev)
        gge.gge_rmsnorm_bwd(dn, h, self.norm, inv, dx, dW=dnorm, dH=dh)
        return dx, dnorm, dw1, dw2


def reference(block, x, r, dy, dh):
    """The same block in fp32 with torch's autograd: (y, dx, dnorm, dw1, dw2)."""
    x = x.float().requires_grad_()
    norm, w1, w2 = (t.float().requires_grad_() for t in (block.norm, block.w1, block.w2))
    h = x + r.float()
    n = h * torch.rsqrt(h.square().mean(1, keepdim=True) + EPS) * norm
    y = torch.nn.functional.silu(n @ w1.t()) @ w2.t()
    grads = torch.autograd.grad((y * dy.float()).sum() + (h * dh.float()).sum(), (x, norm, w1, w2))
    return (y.detach(), *grads)


def relative(a, b):
    return float((a.float() - b).norm() / b.norm())


def run(tokens=512, width=1024, hidden=2048, fmt="mxfp8", seed=0):
    """Relative errors (2-norm) of a training step against fp32 autograd."""
    dev = torch.device("cuda", torch.cuda.current_device())
    block = Block(width, hidden, fmt, dev, seed)
    g = torch.Generator(device=dev).manual_seed(seed + 1)
    x, r, dy, dh = (torch.randn(tokens, width, generator=g, device=dev).bfloat16() for _ in range(4))
    y, _, saved = block.forward(x, r, keep=True)
    out = (y, *block.backward(dy, dh, saved))
    status = gge.gge_read_device_status(dev)
    if status[0] != "GGE_OK":
        raise RuntimeError(f"device status {status}")
    y1, _, _ = block.forward(x[:1], r[:1])   # serving: one token against the same weights
    errors = dict(zip(("y", "dx", "dnorm", "dw1", "dw2"),
                      (relative(a, b) for a, b in zip(out, reference(block, x, r, dy, dh)))))
    errors["one token"] = relative(y1, y[:1].float())
    return errors


if __name__ == "__main__":
    a = sys.argv[1:]
    sizes = [int(v) for v in a[:3]] + [512, 1024, 2048][len(a[:3]):]
    for name, err in run(*sizes, *(a[3:4] or ["mxfp8"])).items():
        print(f"{name:10s} relative error {err:.4f}")
