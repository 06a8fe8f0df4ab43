"""A mixer block with a multi-head selective scan, made of the library's
operators: a joined projection, the short causal convolution, the scan with one
decay a head, the gated group norm and a projection back.

    forward   training and whole prompts, with gradients
    prefill   a prompt (or its next piece), leaving a state to decode from
    step      one token for each of a batch of sequences, states in a pool

Run as a program it checks on the GPU that a prompt taken whole, in pieces and
token by token gives the same outputs, and takes a few training steps:

    python examples/heads_mixer.py
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import scan_selective_fwd_amd as ms  # noqa: E402


class HeadsMixer(torch.nn.Module):
    def __init__(self, width, heads, headdim=64, dstate=128, groups=1, conv_width=4,
                 dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.heads, self.headdim, self.dstate, self.groups = heads, headdim, dstate, groups
        self.inner, self.state_cols = heads * headdim, groups * dstate
        self.conv_cols = self.inner + 2 * self.state_cols
        kw = dict(device=device)
        par = torch.nn.Parameter
        cols = self.inner + self.conv_cols + heads              # z | u, B, C | delta
        self.w_in = par((torch.randn(width, cols, **kw) / math.sqrt(width)).to(dtype))
        self.w_out = par((torch.randn(self.inner, width, **kw) / math.sqrt(self.inner)).to(dtype))
        self.conv_w = par(torch.randn(self.conv_cols, conv_width, **kw) / conv_width)
        self.conv_b = par(torch.zeros(self.conv_cols, **kw))
        self.A = par(-(1 + 15 * torch.rand(heads, **kw)))
        self.D = par(torch.ones(heads, **kw))
        # steps of 0.001 .. 0.1
        step = torch.exp(torch.rand(heads, **kw) * math.log(100) + math.log(0.001))
        self.delta_bias = par(step + torch.log(-torch.expm1(-step)))
        self.norm_w = par(torch.ones(self.inner, **kw))

    def _split(self, row):
        return row.split([self.inner, self.conv_cols, self.heads], -1)

    def _parts(self, y):
        """u, B, C as views of the convolution's rows."""
        u, B, C = y.split([self.inner, self.state_cols, self.state_cols], -1)
        return (u.unflatten(-1, (self.heads, self.headdim)),
                B.unflatten(-1, (self.groups, self.dstate)),
                C.unflatten(-1, (self.groups, self.dstate)))

    def forward(self, x, reset=None):
        """x (batch, L, width); reset: flags of packed sequences."""
        z, xbc, delta = self._split(x @ self.w_in)
        u, B, C = self._parts(ms.conv1d_tokens(xbc, self.conv_w, self.conv_b, reset=reset))
        y = ms.heads_scan(u, delta, self.A, B, C, self.D, self.delta_bias, reset=reset)
        return ms.gated_norm(y.flatten(-2), z, self.norm_w, groups=self.groups) @ self.w_out

    @torch.no_grad()
    def prefill(self, x, cache=None):
        """Returns out and the cache (window, state) after x; `cache`: the one before it."""
        window, state = cache or (None, None)
        z, xbc, delta = self._split(x @ self.w_in)
        y, window = ms.conv1d_tokens_fwd(xbc, self.conv_w, self.conv_b, window=window,
                                         return_window=True)
        u, B, C = self._parts(y)
        y, state = ms.heads_scan_fwd(u, delta, self.A, B, C, self.D, self.delta_bias, state,
                                     return_last_state=True)
        y = ms.gated_norm_fwd(y.flatten(-2), z, self.norm_w, groups=self.groups)
        return y @ self.w_out, (window, state)

    @torch.no_grad()
    def step(self, x, cache, slots=None):
        """One token: x (batch, width); the cache's pool is updated in place at
        `slots` (batch,) int32, or row by row."""
        window, state = cache
        z, xbc, delta = self._split(x @ self.w_in)
        u, B, C = self._parts(ms.conv1d_tokens_update(xbc, window, self.conv_w, self.conv_b,
                                                      slots=slots))
        y = ms.heads_state_update(state, u, delta, self.A, B, C, self.D, self.delta_bias,
                                  slots=slots)
        y = ms.gated_norm_fwd(y.flatten(-2), z, self.norm_w, groups=self.groups)
        return y @ self.w_out


def main():
    torch.manual_seed(0)
    mixer = HeadsMixer(512, heads=16)
    x = torch.randn(2, 300, 512, device="cuda").bfloat16()
    whole = mixer(x).detach()
    a, cache = mixer.prefill(x[:, :200])
    b, cache = mixer.prefill(x[:, 200:290], cache)
    c = [mixer.step(x[:, t], cache) for t in range(290, 300)]
    pieces = torch.cat([a, b, torch.stack(c, 1)], 1)
    far = (pieces.float() - whole.float()).norm() / whole.float().norm()
    print(f"whole against pieces and single tokens: relative difference {float(far):.1e}")

    target = torch.randn_like(x) * 0.1
    opt = torch.optim.AdamW(mixer.parameters(), lr=1e-3)
    losses = []
    for _ in range(5):
        loss = (mixer(x).float() - target.float()).square().mean()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(float(loss.detach()))
    print("training losses:", " ".join(f"{v:.4f}" for v in losses))
    return float(far), losses


if __name__ == "__main__":
    main()
