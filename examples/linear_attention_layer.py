"""A linear attention layer out of the library's operators, as it is used: trained on sequences,
then a prompt in one pass and further tokens one by one.

    python examples/linear_attention_layer.py

One fused projection gives queries, keys and values; prism_qk_norm_rope turns every query and
key head into a unit vector at its position; prism_linattn_forward reads them, and the values
straight out of the projection; prism_linattn_decode_step goes on from the final state.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from linear_recurrent_sequence_causal_gb300 import linattn  # noqa: E402


def angle_table(positions, rotary_dim, base=10000.0, device="cuda"):
    """[positions, rotary_dim] fp32: the cosines, then the sines, of each pair's angle."""
    f = base ** (-torch.arange(0, rotary_dim, 2, device=device, dtype=torch.float64) / rotary_dim)
    a = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], -1).float()


class HeadNorm(torch.autograd.Function):
    """Unit norm and rotation of q and k, with the library's gradient."""

    @staticmethod
    def forward(ctx, q, k, qw, kw, table, positions, seq_lens):
        ctx.how = dict(q_scale=q.shape[-1] ** -0.5, k_scale=q.shape[-1] ** -0.5, eps=1e-6, positions=positions,
                       seq_lens=seq_lens)
        ctx.save_for_backward(q, k, qw, kw, table)
        return linattn.prism_qk_norm_rope(q, k, table, q_weight=qw, k_weight=kw, **ctx.how)

    @staticmethod
    def backward(ctx, dq, dk):
        q, k, qw, kw, table = ctx.saved_tensors
        g = linattn.prism_qk_norm_rope_backward(q, k, table, dq.contiguous(), dk.contiguous(), q_weight=qw,
                                                k_weight=kw, **ctx.how)
        return g["q"], g["k"], g["q_weight"], g["k_weight"], None, None, None


class LinearAttention(torch.autograd.Function):
    """Causal linear attention over a prompt; the state that it ends in has no gradient here."""

    @staticmethod
    def forward(ctx, q, k, v, log_decay, seq_lens):
        ctx.save_for_backward(q, k, v, log_decay, seq_lens)
        out, state = linattn.prism_linattn_forward(q, k, v, log_decay, seq_lens=seq_lens)
        ctx.mark_non_differentiable(state)
        return out, state

    @staticmethod
    def backward(ctx, d_out, _):
        q, k, v, log_decay, seq_lens = ctx.saved_tensors
        g = linattn.prism_linattn_backward(q, k, v, log_decay, d_out.contiguous(), seq_lens=seq_lens)
        return g["q"], g["k"], g["v"], None, None


class Layer(torch.nn.Module):
    def __init__(self, width, heads, head_dim, positions, device="cuda"):
        super().__init__()
        self.heads, self.head_dim = heads, head_dim
        kw = dict(device=device, dtype=torch.bfloat16)
        self.qkv = torch.nn.Linear(width, 3 * heads * head_dim, bias=False, **kw)
        self.out = torch.nn.Linear(heads * head_dim, width, bias=False, **kw)
        self.q_weight = torch.nn.Parameter(torch.ones(head_dim, device=device))
        self.k_weight = torch.nn.Parameter(torch.ones(head_dim, device=device))
        # from a memory of a few tokens to one of a few thousand
        slope = torch.logspace(-0.3, -3.3, heads, device=device)
        self.register_buffer("log_decay", -slope)
        self.register_buffer("table", angle_table(positions, head_dim, device=device))

    def split(self, x):
        B, T, _ = x.shape
        qkv = self.qkv(x).view(B, T, 3, self.heads, self.head_dim)
        return qkv[:, :, 0], qkv[:, :, 1], qkv[:, :, 2]

    def forward(self, x, seq_lens=None):
        """x [B,T,width] -> ([B,T,width], state): a prompt, or a batch to train on."""
        q, k, v = self.split(x)
        q, k = HeadNorm.apply(q, k, self.q_weight, self.k_weight, self.table, None, seq_lens)
        o, state = LinearAttention.apply(q, k, v, self.log_decay, seq_lens)
        return self.out(o.flatten(2)), state

    @torch.no_grad()
    def step(self, x, state, positions):
        """x [B,width], one token of each sequence at its position [B]; state moves on in place."""
        q, k, v = self.split(x[:, None])
        q, k = HeadNorm.apply(q, k, self.q_weight, self.k_weight, self.table, positions[:, None], None)
        o = linattn.prism_linattn_decode_step(q[:, 0], k[:, 0], v[:, 0], self.log_decay, state)
        return self.out(o.flatten(1))


def main():
    torch.manual_seed(0)
    B, T, width, new = 4, 300, 256, 8
    layer = Layer(width, heads=4, head_dim=64, positions=T + new)
    x = torch.randn(B, T + new, width, device="cuda", dtype=torch.bfloat16)
    lens = torch.tensor([T, T, 17, 0], device="cuda", dtype=torch.int32)

    # train: each token's output towards the mean of the tokens up to it
    want = x[:, :T].float().cumsum(1) / torch.arange(1, T + 1, device="cuda")[:, None]
    live = (torch.arange(T, device="cuda") < lens[:, None])[..., None]
    opt = torch.optim.Adam(layer.parameters(), lr=1e-3)
    losses = []
    for _ in range(30):
        y, _ = layer(x[:, :T], lens)
        loss = ((y.float() - want) * live).square().sum() / live.sum()
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    print(f"loss {losses[0]:.3f} -> {losses[-1]:.3f}")

    # serve: a prompt, then token by token; the same as the whole sequence at once
    with torch.no_grad():
        whole, _ = layer(x)
        y, state = layer(x[:, :T])
        off = []
        for t in range(T, T + new):
            y = layer.step(x[:, t], state, torch.full((B,), t, device="cuda", dtype=torch.int32))
            off.append(((y - whole[:, t]).float().norm() / whole[:, t].float().norm()).item())
    print(f"tokens after the prompt differ from the whole pass by {max(off):.1e} of their norm")
    return losses, off


if __name__ == "__main__":
    main()
