"""A linear attention layer with a fixed decay per head, trained for some steps and then used as a
language model serves it: prompts of unequal lengths in one batch, then token by token.

    y = (group_norm(linear_attention(x Wq, x Wk, x Wv)) * silu(x Wz)) Wo

    python examples/linear_attention_layer.py        (needs the GPU and the built library)
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_31_gb300 as gdr  # noqa: E402
from gated_delta_rule_31_gb300.autograd import group_norm, linear_attention  # noqa: E402


class LinearAttentionLayer(torch.nn.Module):
    def __init__(self, width, key_heads, value_heads, key_dim, value_dim, dtype=torch.bfloat16, device="cuda"):
        super().__init__()
        self.shape = key_heads, value_heads, key_dim, value_dim

        def weight(n_in, n_out):
            return torch.nn.Parameter(torch.randn(n_in, n_out, device=device).mul_(n_in ** -0.5).to(dtype))

        self.wq, self.wk = weight(width, key_heads * key_dim), weight(width, key_heads * key_dim)
        self.wv, self.wz = weight(width, value_heads * value_dim), weight(width, value_heads * value_dim)
        self.wo = weight(value_heads * value_dim, width)
        self.norm = torch.nn.Parameter(torch.ones(value_heads * value_dim, device=device))
        # half-lives from about a token to hundreds of tokens over the heads
        self.register_buffer("decay", -torch.exp2(-torch.linspace(0.5, 9.0, value_heads, device=device)))

    def _project(self, x):
        hk, hv, dk, dv = self.shape
        lead = x.shape[:-1]
        return (x @ self.wq).view(*lead, hk, dk), (x @ self.wk).view(*lead, hk, dk), (x @ self.wv).view(*lead, hv, dv)

    def forward(self, x, state=None, lengths=None):
        """x [B, T, width], in training or for a prompt: (y, the state after each row's last token)."""
        o, state = linear_attention(*self._project(x), self.decay, state, lengths=lengths)
        n = group_norm(o.flatten(2), self.shape[1], self.norm, gate=x @ self.wz, activation="silu")
        return n @ self.wo, state

    @torch.no_grad()
    def step(self, x, state):
        """x [B, width], one token of each sequence; the state is updated in place."""
        o = gdr.linear_decode_step(*self._project(x), self.decay, state)
        n = gdr.group_norm_fwd(o.flatten(1), self.shape[1], self.norm, gate=x @ self.wz, activation="silu")
        return n @ self.wo


def main(steps=30):
    """Trains the layer to repeat the token before, then decodes and compares with one long prompt. Returns
    (first loss, last loss, the largest difference of a decoded output)."""
    torch.manual_seed(0)
    B, T, width = 4, 300, 256
    layer = LinearAttentionLayer(width, key_heads=2, value_heads=4, key_dim=64, value_dim=64)
    x = torch.randn(B, T, width, device="cuda", dtype=torch.bfloat16)
    optimizer = torch.optim.Adam(layer.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        y, _ = layer(x)
        loss = (y[:, 1:].float() - x[:, :-1].float()).square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(float(loss.detach()))

    with torch.no_grad():
        n, more = [200, 1, 129, 77], 40  # prompts of unequal lengths, then 40 tokens each
        lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
        _, state = layer(x, lengths=lengths)
        at = lengths.long()
        rows = torch.arange(B, device="cuda")
        out = []
        for i in range(more):
            out.append(layer.step(x[rows, at + i], state))
        whole, _ = layer(x)
        off = max(float((out[i][b] - whole[b, n[b] + i]).abs().max()) for b in range(B) for i in range(more))
    return losses[0], losses[-1], off


if __name__ == "__main__":
    first, last, off = main()
    print(f"loss {first:.3f} -> {last:.3f}; decoded outputs differ from the whole sequence's by at most {off:.3g}")
