"""A small upsampling decoder from the library's operators: trained on whole sequences, then streamed frame by frame.

Frames [B, T, C] pass a causal mixer (RMS norm, linear attention with a decay for each head), a gated feed-forward layer and a
transposed convolution that turns each frame into `stride` samples, as in a vocoder.  The matrix products between them are torch's.
Training keeps the feed-forward layer's and the convolution's inputs as 8-bit checkpoints; streaming carries one state of constant
size instead of a cache that grows.

    python examples/upsampling_decoder.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import transposed_convolution_convtranspose1_gb300 as ct  # noqa: E402


class Decoder:
    def __init__(self, channels=256, heads=4, hidden=512, samples=16, stride=4, dtype=torch.bfloat16, device="cuda", seed=0):
        g = torch.Generator().manual_seed(seed)

        def weight(*shape, fan):
            return (torch.randn(shape, generator=g) * fan ** -0.5).to(device, dtype).requires_grad_()

        self.heads, self.size, self.stride = heads, channels // heads, stride
        self.norms = [torch.ones(channels, dtype=dtype, device=device, requires_grad=True) for _ in range(3)]
        self.qkv, self.mix = weight(channels, 3 * channels, fan=channels), weight(channels, channels, fan=channels)
        self.gate_up, self.down = weight(channels, 2 * hidden, fan=channels), weight(hidden, channels, fan=hidden)
        self.conv = weight(channels, samples, 2 * stride, fan=2 * channels)
        self.bias = torch.zeros(samples, dtype=dtype, device=device, requires_grad=True)
        # memories of 2 to 256 frames
        self.log_decay = -torch.exp2(-1.0 - 7.0 * torch.arange(heads, device=device) / max(1, heads - 1)).float()

    def parameters(self):
        return self.norms + [self.qkv, self.mix, self.gate_up, self.down, self.conv, self.bias]

    def _heads(self, y):
        q, k, v = (y @ self.qkv).unflatten(-1, (3, self.heads, self.size)).unbind(2)  # slices of one projection, no copies
        return q, k, v

    def train_forward(self, x, lengths=None):
        """[B, T, C] -> samples [B, samples, T * stride], recorded for autograd."""
        o, _ = ct.linear_attention_autograd(*self._heads(ct.rms_norm_autograd(x, self.norms[0])), self.log_decay, lengths=lengths)
        y, h = ct.rms_norm_autograd(o.flatten(2) @ self.mix, self.norms[1], x)
        gate, up = (y @ self.gate_up).chunk(2, -1)
        z = ct.checkpointed_activation_autograd(gate, up, "silu", quant="int8")
        y, _ = ct.rms_norm_autograd(z @ self.down, self.norms[2], h)
        return ct.conv_transpose_autograd(y.transpose(1, 2).contiguous(), self.conv, self.bias, stride=self.stride,
                                          padding=self.stride // 2, checkpoint="int8")

    @torch.no_grad()
    def frames(self, x, state):
        """Features of one or more new frames; `state` [B, H, D, D] is carried in place."""
        o, _ = ct.linear_attention(*self._heads(ct.rms_norm(x, self.norms[0])[0]), self.log_decay, state, state_out=state)
        y, h, _, _ = ct.rms_norm(o.flatten(2) @ self.mix, self.norms[1], x)
        gate, up = (y @ self.gate_up).chunk(2, -1)
        z, _, _ = ct.checkpointed_activation(gate, up, "silu")
        return ct.rms_norm(z @ self.down, self.norms[2], h)[0]

    @torch.no_grad()
    def samples(self, y):
        return ct.conv_transpose(y.transpose(1, 2).contiguous(), self.conv, self.bias, stride=self.stride, padding=self.stride // 2)

    def new_state(self, batch):
        return torch.zeros(batch, self.heads, self.size, self.size, device=self.log_decay.device)


def main(steps=30, B=4, T=200):
    torch.manual_seed(0)
    model = Decoder()
    x = torch.randn(B, T, 256, device="cuda").bfloat16()
    target = torch.randn(B, 16, 1, device="cuda").expand(B, 16, T * 4).bfloat16()
    optimizer = torch.optim.Adam(model.parameters(), lr=1e-3)
    losses = []
    for _ in range(steps):
        loss = (model.train_forward(x) - target).float().square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.item())
    whole = model.train_forward(x).detach()
    # a prompt of 150 frames, then one frame at a time
    state = model.new_state(B)
    parts = [model.frames(part.contiguous(), state) for part in [x[:, :150], *x[:, 150:].split(1, 1)]]
    streamed = model.samples(torch.cat(parts, 1))
    off = (streamed.float() - whole.float()).norm() / whole.float().norm()
    return losses, off.item()


if __name__ == "__main__":
    losses, off = main()
    print("loss %.4f -> %.4f; streamed against whole: relative difference %.1e" % (losses[0], losses[-1], off))
