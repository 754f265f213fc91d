"""A training step and a serving call of a small model over item histories,
with the token operators together:

    x      = sqrt(dim) * table[token]                     emb_lookup_scaled
    q, s   = int8 codes of norm(x + position) * weight    rms_norm_residual_i8
    p      = sigmoid((q s) (w8 w_scale)^T + bias)         linear_i8_bias_act
    table -= rate * d loss / d table                      emb_lookup_grad, in place

The dense layer is held in int8 and stays as it is; the table is what the step
learns.  The loss is the mean binary cross entropy of p against which classes
follow a token; its gradient passes the codes as if they were not rounded.

    python examples/token_step.py [steps]                 (needs the GPU)
"""
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

EPS = 1e-6


class HistoryModel:
    """Tables and quantised layer on the current GPU, made from a seed."""

    def __init__(self, rows=5000, dim=96, length=20, classes=64, seed=0):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape):
            return torch.randn(shape, generator=g, device="cuda")

        self.rows, self.dim, self.length, self.classes = rows, dim, length, classes
        self.scale = math.sqrt(dim)
        self.table = normal(rows, dim) * 0.05
        self.position = normal(length, dim) * 0.1
        self.weight = 1.0 + 0.1 * normal(dim)
        w = normal(classes, dim) / math.sqrt(dim)
        self.w_scale = w.abs().amax(1) / 127.0
        self.w8 = torch.round(w / self.w_scale[:, None]).to(torch.int8)
        self.bias = normal(classes) * 0.1

    def forward(self, tokens):
        """tokens (batch, length) int32, -1 where a history is shorter: the
        probabilities (batch * length, classes) and the normed rows' h."""
        import dlrm_embedding_bag_amd as fw
        x = fw.emb_lookup_scaled(self.table, tokens, self.scale).view(-1, self.dim)
        position = self.position[:tokens.shape[1]].repeat(tokens.shape[0], 1)
        h, q, s = fw.rms_norm_residual_i8(x, self.weight, position, eps=EPS)
        return fw.linear_i8_bias_act(q, s, self.w8, self.w_scale, self.bias, "sigmoid"), h

    def table_gradient_rows(self, p, h, target):
        """d loss / d (sqrt(dim) * table[token]), one row for each token."""
        dz = (p - target) / p.numel()
        dy = (dz @ (self.w8.float() * self.w_scale[:, None])) * self.weight
        r = (h.square().mean(1, keepdim=True) + EPS).rsqrt()
        return r * dy - h * (r ** 3) * (h * dy).mean(1, keepdim=True)

    def step(self, tokens, target, rate):
        """One step of gradient descent on the table; the loss before it."""
        import torch

        import dlrm_embedding_bag_amd as fw
        p, h = self.forward(tokens)
        loss = torch.nn.functional.binary_cross_entropy(p, target)
        fw.emb_lookup_grad(self.table_gradient_rows(p, h, target), tokens.view(-1),
                           scale=-rate * self.scale, out=self.table, accumulate=True)
        return loss

    def serve(self, tokens, position):
        """Probabilities after one more token of each request: tokens (batch,)."""
        import dlrm_embedding_bag_amd as fw
        x = fw.emb_lookup_scaled(self.table, tokens, self.scale)
        _, q, s = fw.rms_norm_residual_i8(x, self.weight,
                                          self.position[position].expand(len(tokens), -1), eps=EPS)
        return fw.linear_i8_bias_act(q, s, self.w8, self.w_scale, self.bias, "sigmoid")


def batch_of(model, batch, seed=1):
    """Histories whose next classes depend on the item: (tokens, target)."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    tokens = torch.randint(0, model.rows, (batch, model.length), generator=g, device="cuda",
                           dtype=torch.int32)
    short = torch.rand(batch, model.length, generator=g, device="cuda") < 0.05
    tokens = torch.where(short, torch.full_like(tokens, -1), tokens)
    classes = torch.arange(model.classes, device="cuda")
    target = ((tokens.view(-1, 1) * 31 + classes * 17) % 7 < 2).float()
    return tokens, target


def main(steps=30):
    model = HistoryModel()
    tokens, target = batch_of(model, 256)
    for i in range(steps):
        loss = model.step(tokens, target, rate=2000.0)
        if i % 10 == 0 or i + 1 == steps:
            print(f"step {i}: loss {loss.item():.4f}", flush=True)
    p = model.serve(tokens[:8, 0].contiguous(), 0)
    print(f"served {tuple(p.shape)}, mean probability {p.mean().item():.4f}", flush=True)


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 30)
