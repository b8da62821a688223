"""A residual MLP block in 8 bits with a scale for each block of 128, from pre-norm to weight
gradients: one forward pass for serving and one training step that keeps nothing in 16 bits but
the residual stream.

    x, r  --gge_layernorm-->  h = x + r (16 bits, and 8 for the backward),  codes of n = norm(h)
    codes, W1  --gge_gemm_b128-->  u (8 bits, kept),  codes of a = gelu(u)
    codes, W2  --gge_gemm_b128-->  y

Backward.  Weights have a scale for each block of 128 x 128, so their transposes hold the same
blocks; activations are turned in 8 bits, with new scales along the tokens:

    da = dy W2, du = gelu'(u) da in 8 bits  (gge_gemm_b128_dact)         dn = du W1
    dW2 += dy^T a      dW1 += du^T n      (fp32, added to in place)
    dn, h in 8 bits  --gge_layernorm_bwd-->  the gradient of x and r, and of weight and bias

    python examples/block_scaled_mlp.py [tokens] [width] [hidden]
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from grouped_gemm_epilogues_gb300 import binding as gge  # noqa: E402

EPS = 1e-5


def quantised(x, block_rows=1):
    """x (rows, cols; a transposed view is fine) in 8 bits."""
    q = gge.b128_empty(x.shape[0], x.shape[1], block_rows, device=x.device)
    gge.gge_b128_quantize(x, q)
    return q


def turned(q):
    """q's numbers transposed, quantised along their new rows."""
    t = gge.b128_empty(q.codes.shape[1], q.codes.shape[0], device=q.codes.device)
    gge.gge_b128_transpose(q, t)
    return t


class Block:
    """Weights as a program keeps them: bf16 masters, their codes laid out once, fp32 gradients."""

    def __init__(self, width, hidden, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)

        def draw(*shape, scale):
            return (torch.randn(*shape, generator=g, device=device) * scale).bfloat16()

        self.width, self.hidden = width, hidden
        self.weight = 1 + draw(width, scale=0.1)
        self.bias = draw(width, scale=0.1)
        self.w1, self.w2 = draw(hidden, width, scale=width ** -0.5), draw(width, hidden, scale=hidden ** -0.5)
        self.dw1, self.dw2 = torch.zeros(hidden, width, device=device), torch.zeros(width, hidden, device=device)
        self.refresh()

    def refresh(self):
        """The codes of the weights, after an update."""
        self.q1, self.q2 = quantised(self.w1, 128), quantised(self.w2, 128)
        self.q1t, self.q2t = quantised(self.w1.t(), 128), quantised(self.w2.t(), 128)

    def forward(self, x, r, keep=False):
        tokens, dev = x.shape[0], x.device
        h = torch.empty_like(x)
        mean, rstd = torch.empty(tokens, device=dev), torch.empty(tokens, device=dev)
        n = gge.b128_empty(tokens, self.width, device=dev)
        h8 = gge.b128_empty(tokens, self.width, device=dev) if keep else None
        gge.gge_layernorm(x, self.weight, self.bias, residual=r, residual_out=h, Q=n, H8=h8, mean=mean, rstd=rstd, eps=EPS)
        u = gge.b128_empty(tokens, self.hidden, device=dev) if keep else None
        a = gge.b128_empty(tokens, self.hidden, device=dev)
        gge.gge_gemm_b128(n, self.q1, D=u, PostAct=a, act="gelu_tanh")
        y = torch.empty_like(x)
        gge.gge_gemm_b128(a, self.q2, D=y)
        return y, h, (h8, mean, rstd, n, u, a) if keep else None

    def backward(self, dy, dh, saved):
        h8, mean, rstd, n, u, a = saved
        dev = dy.device
        tokens = dy.shape[0]
        du = gge.b128_empty(tokens, self.hidden, device=dev)
        q_dy = quantised(dy)
        gge.gge_gemm_b128_dact(q_dy, self.q2t, u, du, "gelu_tanh")
        dn = torch.empty_like(dy)
        gge.gge_gemm_b128(du, self.q1t, D=dn)
        gge.gge_gemm_b128(turned(q_dy), turned(a), D=self.dw2, C=self.dw2)
        gge.gge_gemm_b128(turned(du), turned(n), D=self.dw1, C=self.dw1)
        dx = torch.empty_like(dy)
        dweight, dbias = torch.empty(self.width, device=dev), torch.empty(self.width, device=dev)
        gge.gge_layernorm_bwd(dn, h8, self.weight, mean, rstd, dx, dW=dweight, dB=dbias, dH=dh)
        return dx, dweight, dbias


def reference(block, x, r, dy, dh):
    """The same block in fp32 with torch's autograd: (y, dx, dweight, dbias, dw1, dw2)."""
    x = x.float().requires_grad_()
    weight, bias, w1, w2 = (t.float().requires_grad_() for t in (block.weight, block.bias, block.w1, block.w2))
    h = x + r.float()
    n = torch.nn.functional.layer_norm(h, (block.width,), weight, bias, EPS)
    y = torch.nn.functional.gelu(n @ w1.t(), approximate="tanh") @ w2.t()
    grads = torch.autograd.grad((y * dy.float()).sum() + (h * dh.float()).sum(), (x, weight, bias, w1, w2))
    return (y.detach(), *grads)


def relative(a, b):
    return float((a.float() - b).norm() / b.norm())


def run(tokens=512, width=1024, hidden=2048, seed=0):
    """Relative errors (2-norm) of a training step against fp32 autograd."""
    dev = torch.device("cuda", torch.cuda.current_device())
    block = Block(width, hidden, dev, seed)
    g = torch.Generator(device=dev).manual_seed(seed + 1)
    x, r, dy, dh = (torch.randn(tokens, width, generator=g, device=dev).bfloat16() for _ in range(4))
    y, _, saved = block.forward(x, r, keep=True)
    out = (y, *block.backward(dy, dh, saved), block.dw1, block.dw2)
    status = gge.gge_read_device_status(dev)
    if status[0] != "GGE_OK":
        raise RuntimeError(f"device status {status}")
    y1, _, _ = block.forward(x[:1], r[:1])   # serving: one token against the same weights
    errors = dict(zip(("y", "dx", "dweight", "dbias", "dw1", "dw2"),
                      (relative(a, b) for a, b in zip(out, reference(block, x, r, dy, dh)))))
    errors["one token"] = relative(y1, y[:1].float())
    return errors


if __name__ == "__main__":
    a = [int(v) for v in sys.argv[1:]]
    for name, err in run(*(a + [512, 1024, 2048][len(a):])).items():
        print(f"{name:10s} relative error {err:.4f}")
