"""A residual block whose mixer is the gated linear recurrence, made of the library's
operators: the norm with the residual's addition, a joined projection, the short
causal convolution, the gates' projection, the recurrence under its gate, and a
projection back.

    forward   training and whole prompts, with gradients
    prefill   a prompt (or its next piece), leaving a cache to decode from
    step      one token for each of a batch of sequences, states in pools

Each call takes the last block's output x and the residual stream, and returns its own
output and the stream with x added.  Run as a program it checks on the GPU that a
prompt taken whole, in pieces and token by token gives the same outputs, and takes a
few training steps:

    python examples/recurrent_block.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import scan_selective_fwd_amd as ms  # noqa: E402


class RecurrentBlock(torch.nn.Module):
    def __init__(self, width, inner, conv_width=4, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.inner = inner
        kw = dict(device=device)
        par = torch.nn.Parameter
        mat = lambda a, b: par((torch.randn(a, b, **kw) / math.sqrt(a)).to(dtype))  # noqa: E731
        self.norm_w = par(torch.ones(width, **kw))
        self.w_in = mat(width, 2 * inner)                       # z | x
        self.conv_w = par(torch.randn(inner, conv_width, **kw) / conv_width)
        self.conv_b = par(torch.zeros(inner, **kw))
        self.w_gates = mat(inner, 2 * inner)                    # r | i
        # channels that keep 0.9 .. 0.999 of their state at an eighth of the gate
        self.log_keep = par(torch.log(-8 * torch.log(0.9 + 0.099 * torch.rand(inner, **kw))))
        self.w_out = mat(inner, width)

    @property
    def A(self):
        return -torch.exp(self.log_keep)

    def _gates(self, x):
        return (x @ self.w_gates).split([self.inner, self.inner], -1)

    def forward(self, x, stream, reset=None):
        """x (batch, L, width), stream of x's type or float32; reset: flags of packed
        sequences."""
        y, stream = ms.residual_norm(x, stream, self.norm_w)
        z, u = (y @ self.w_in).split([self.inner, self.inner], -1)
        u = ms.conv1d_tokens(u, self.conv_w, self.conv_b, reset=reset)
        h = ms.gated_recurrence(u, *self._gates(u), self.A, z, reset=reset)
        return h @ self.w_out, stream

    @torch.no_grad()
    def prefill(self, x, stream, cache=None):
        """Returns out, the stream and the cache (window, state) after x; `cache`: the
        one before it."""
        window, state = cache or (None, None)
        y, stream = ms.residual_norm_fwd(x, stream, self.norm_w)
        z, u = (y @ self.w_in).split([self.inner, self.inner], -1)
        u, window = ms.conv1d_tokens_fwd(u, self.conv_w, self.conv_b, window=window,
                                         return_window=True)
        h, state = ms.gated_recurrence_fwd(u, *self._gates(u), self.A, z, state,
                                           return_last_state=True)
        return h @ self.w_out, stream, (window, state)

    @torch.no_grad()
    def step(self, x, stream, cache, slots=None):
        """One token: x, stream (batch, width); the stream is carried on in place, and
        the cache's pools are updated in place at `slots` (batch,) int32, or row by row."""
        window, state = cache
        y, stream = ms.residual_norm_fwd(x, stream, self.norm_w, residual_out=stream)
        z, u = (y @ self.w_in).split([self.inner, self.inner], -1)
        u = ms.conv1d_tokens_update(u, window, self.conv_w, self.conv_b, slots=slots)
        h = ms.gated_recurrence_update(state, u, *self._gates(u), self.A, z, slots=slots)
        return h @ self.w_out, stream


def main():
    torch.manual_seed(0)
    block = RecurrentBlock(512, 768)
    x = torch.randn(2, 700, 512, device="cuda").bfloat16()
    stream = torch.randn(2, 700, 512, device="cuda")
    whole = block(x, stream)[0].detach()
    a, _, cache = block.prefill(x[:, :400], stream[:, :400])
    b, _, cache = block.prefill(x[:, 400:690], stream[:, 400:690], cache)
    c = [block.step(x[:, t], stream[:, t].contiguous(), cache)[0] for t in range(690, 700)]
    pieces = torch.cat([a, b, torch.stack(c, 1)], 1)
    far = (pieces.float() - whole.float()).norm() / whole.float().norm()
    print(f"whole against pieces and single tokens: relative difference {float(far):.1e}")

    target = torch.randn_like(stream) * 0.1
    opt = torch.optim.AdamW(block.parameters(), lr=1e-3)
    losses = []
    for _ in range(5):
        out, kept = block(x, stream)
        loss = (out.float() + kept - stream - target).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    print("training losses:", " ".join(f"{v:.4f}" for v in losses))
    return float(far), losses


if __name__ == "__main__":
    main()
