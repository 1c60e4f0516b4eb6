"""A feed-forward layer of a transformer: one training step in bf16 and one serving step in 8 bits.

    python examples/feed_forward.py

Training: h = x + residual, n = norm(h), u = gelu(n·W1ᵀ + b1), out = u·W2ᵀ + h, and its gradients.
Serving:  the same layer with e4m3 weights, the norm quantising its rows for the product that
follows, for a prompt and for a single token.
Both are compared with the formulas in 64 bits.
"""

import math
import os
import sys

import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))
import tile_level_gemm_amd as tg  # noqa: E402


class FeedForward:
    def __init__(self, width, hidden, generator):
        def randn(*shape):
            return torch.randn(shape, generator=generator, device="cuda")
        self.norm = (1 + 0.1 * randn(width)).bfloat16()
        self.w1 = (randn(hidden, width) / math.sqrt(width)).bfloat16()
        self.b1 = (0.1 * randn(hidden)).bfloat16()
        self.w2 = (randn(width, hidden) / math.sqrt(hidden)).bfloat16()
        # 8-bit weights with one scale per output column, as a serving checkpoint holds them
        self.w1_8, self.s1 = self.quantise(self.w1)

    @staticmethod
    def quantise(w):
        s = w.float().abs().amax(dim=1) / 448
        return (w.float() / s[:, None]).to(torch.float8_e4m3fn), s

    def forward(self, x, residual):
        n = tg.rms_norm(x, self.norm, residual=residual)
        u, z = tg.gemm_ep(n.y, self.w1, bias=self.b1, act="gelu", keep_z=True)
        return tg.gemm_ep(u, self.w2, residual=n.h), (n, u, z)

    def backward(self, dout, saved):
        """Gradients of norm, w1, b1, w2 and of x (which is also the residual's)."""
        n, u, z = saved
        _, du, dw2, _ = tg.gemm_ep_backward(dout, u, self.w2, need_dbias=False)
        _, dn, dw1, db1 = tg.gemm_ep_backward(du, n.y, self.w1, Z=z, act="gelu")
        dx, dnorm = tg.rms_norm_backward(dn, n.h, self.norm, n.rstd, dH=dout)
        return dict(norm=dnorm, w1=dw1, b1=db1, w2=dw2, x=dx)

    def serve(self, x, residual):
        n = tg.rms_norm(x, self.norm, residual=residual, scales="row")
        u = tg.gemm_ep(n.y, self.w1_8, row_scale=n.scale, col_scale=self.s1, bias=self.b1, act="gelu")
        return tg.gemm_ep(u, self.w2, residual=n.h)


def reference(layer, x, residual, dout=None):
    """The same in 64 bits; the sum is rounded as the residual stream is held."""
    p = {k: getattr(layer, k).double().requires_grad_() for k in ("norm", "w1", "b1", "w2")}
    h = (x.float() + residual.float()).to(x.dtype).double().requires_grad_()
    y = h * torch.rsqrt(h.square().mean(dim=1, keepdim=True) + 1e-5) * p["norm"]
    z = y @ p["w1"].t() + p["b1"]
    out = 0.5 * z * torch.special.erfc(-z / math.sqrt(2)) @ p["w2"].t() + h
    if dout is None:
        return out.detach()
    grads = torch.autograd.grad(out, [h, *p.values()], dout.double())
    return out.detach(), dict(zip(["x", *p], grads))


def off(got, want):
    return float((got.double() - want).norm() / want.norm())


def main(width=1024, hidden=4096, tokens=512):
    g = torch.Generator(device="cuda").manual_seed(0)
    layer = FeedForward(width, hidden, g)
    x, residual, dout = (torch.randn(tokens, width, generator=g, device="cuda").bfloat16() for _ in range(3))
    out, saved = layer.forward(x, residual)
    grads = layer.backward(dout, saved)
    want, wants = reference(layer, x, residual, dout)
    worst = {"out": off(out, want), **{k: off(grads[k], wants[k]) for k in wants}}
    print("training, relative error:", ", ".join(f"{k} {v:.1e}" for k, v in worst.items()))
    served = {n: off(layer.serve(x[:n], residual[:n]), want[:n]) for n in (tokens, 1)}
    print("serving in 8 bits, relative error:", ", ".join(f"{n} tokens {v:.1e}" for n, v in served.items()))
    # bf16 keeps 2^-8 of each value held on the way; e4m3 rounds the norm and the weights to 2^-4
    assert max(worst.values()) < 2.0 ** -6 and max(served.values()) < 2.0 ** -4
    return worst, served


if __name__ == "__main__":
    main()
