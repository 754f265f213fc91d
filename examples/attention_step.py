"""A training step and serving calls of a small model over item histories with
attention, the attention operators beside the token operators:

    x       = sqrt(dim) * table[token]                 emb_lookup_scaled
    q, k    = turned norms of x Wq, x Wk               qk_norm_rope
    a       = causal attention within each history     attention_packed
    p       = sigmoid((x + a Wo) Wc)

and back through attention_packed_grad, qk_norm_rope_grad and emb_lookup_grad to
every weight and the table.  Histories are packed: no row is padding.  When
serving, each new item's keys and values go into a paged cache in 8 or 4 bits
(kv_cache_write) and its query reads the history from there (attention_cached).

    python examples/attention_step.py [steps]                 (needs the GPU)
"""
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

EPS = 1e-6


class AttentionModel:
    """Weights on the current GPU, made from a seed."""

    def __init__(self, rows=5000, dim=64, heads=4, kv_heads=2, head=32, classes=64, seed=0):
        import torch
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale=1.0):
            return torch.randn(shape, generator=g, device="cuda") * scale

        self.rows, self.dim, self.heads, self.kv_heads, self.head = rows, dim, heads, kv_heads, head
        self.scale = math.sqrt(dim)
        self.freqs = 10000.0 ** (-torch.arange(head // 2, device="cuda") / (head // 2))
        self.weights = {
            "table": normal(rows, dim, scale=0.1),
            "qkv": normal(dim, (heads + 2 * kv_heads) * head, scale=dim ** -0.5),
            "q_norm": 1.0 + normal(head, scale=0.1), "k_norm": 1.0 + normal(head, scale=0.1),
            "out": normal(heads * head, dim, scale=(heads * head) ** -0.5),
            "classes": normal(dim, classes, scale=dim ** -0.5)}

    def _heads(self, tokens, positions):
        """x, and q, k, v with q and k before and after norm and rotation."""
        import dlrm_embedding_bag_amd as fw
        w = self.weights
        x = fw.emb_lookup_scaled(w["table"], tokens, self.scale)
        qkv = (x @ w["qkv"]).view(len(tokens), -1, self.head)
        q, k, v = qkv.split((self.heads, self.kv_heads, self.kv_heads), 1)
        qn, kn = fw.qk_norm_rope(q, k, positions, self.freqs, w["q_norm"], w["k_norm"], eps=EPS)
        return x, q, k, v, qn, kn

    def _answer(self, x, a):
        import torch
        y = x + a.reshape(len(x), -1) @ self.weights["out"]
        return y, torch.sigmoid(y @ self.weights["classes"])

    def forward(self, tokens, positions, offsets):
        """Probabilities of each token's classes; histories offsets[b]:offsets[b + 1]."""
        import dlrm_embedding_bag_amd as fw
        x, _, _, v, qn, kn = self._heads(tokens, positions)
        a, _ = fw.attention_packed(qn, kn, v, offsets)
        return self._answer(x, a)[1]

    def gradients(self, tokens, positions, offsets, target):
        """The loss (mean binary cross entropy) and its gradients by weight."""
        import torch

        import dlrm_embedding_bag_amd as fw
        w = self.weights
        x, q, k, v, qn, kn = self._heads(tokens, positions)
        a, lse = fw.attention_packed(qn, kn, v, offsets)
        y, p = self._answer(x, a)
        loss = torch.nn.functional.binary_cross_entropy(p, target)
        dz = (p - target) / p.numel()
        dy = dz @ w["classes"].T
        flat = a.reshape(len(x), -1)
        grads = {"classes": y.T @ dz, "out": flat.T @ dy}
        da = (dy @ w["out"].T).view_as(a)
        dqn, dkn, dv = fw.attention_packed_grad(da, qn, kn, v, a, lse, offsets)
        dq, dk, grads["q_norm"], grads["k_norm"] = fw.qk_norm_rope_grad(
            dqn, dkn, q, k, positions, self.freqs, w["q_norm"], w["k_norm"], eps=EPS)
        dqkv = torch.cat((dq, dk, dv), 1).view(len(x), -1)
        grads["qkv"] = x.T @ dqkv
        grads["table"] = fw.emb_lookup_grad(dy + dqkv @ w["qkv"].T, tokens, self.rows,
                                            scale=self.scale)
        return loss, grads

    def step(self, tokens, positions, offsets, target, rate):
        loss, grads = self.gradients(tokens, positions, offsets, target)
        for name, g in grads.items():
            self.weights[name].sub_(g, alpha=rate)
        return loss


class Server:
    """Histories that grow by one item a call, kept in a cache of `bits` bits.
    Request b has the pages b, b + batch, b + 2 batch, ..."""

    def __init__(self, model, batch, longest, bits=8, page=16):
        import torch

        import dlrm_embedding_bag_amd as fw
        each = -(-longest // page)
        self.model, self.batch, self.page = model, batch, page
        self.cache = fw.kv_cache(batch * each, page, model.kv_heads, model.head, bits)
        self.requests = torch.arange(batch, device="cuda", dtype=torch.int32)
        self.table = (self.requests[:, None]
                      + batch * torch.arange(each, device="cuda", dtype=torch.int32))
        self.lengths = torch.zeros(batch, device="cuda", dtype=torch.int32)

    def next(self, tokens):
        """Probabilities after one more item of each request: tokens (batch,)."""
        import dlrm_embedding_bag_amd as fw
        m, at = self.model, self.lengths.clone()
        x, _, _, v, qn, kn = m._heads(tokens, at)
        page = self.table[self.requests.long(), (at // self.page).long()]
        fw.kv_cache_write(self.cache, kn, v, page * self.page + at % self.page)
        self.lengths += 1
        a = fw.attention_cached(qn, self.cache, self.table, self.lengths)
        return m._answer(x, a)[1]


def batch_of(model, batch, longest, classes, seed=1):
    """Histories of 1 .. longest items whose next classes depend on the item and on
    the history's first: (tokens, positions, offsets, target), packed."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    lengths = torch.randint(1, longest + 1, (batch,), generator=g, device="cuda")
    offsets = torch.cat((lengths.new_zeros(1), lengths.cumsum(0)))
    n = int(offsets[-1])
    which = torch.repeat_interleave(torch.arange(batch, device="cuda"), lengths)
    positions = (torch.arange(n, device="cuda") - offsets[which]).to(torch.int32)
    tokens = torch.randint(0, model.rows, (n,), generator=g, device="cuda", dtype=torch.int32)
    first = tokens[offsets[which]]
    c = torch.arange(classes, device="cuda")
    target = (((tokens + first)[:, None] * 31 + c * 17) % 7 < 2).float()
    return tokens, positions, offsets.to(torch.int32), target


def main(steps=30):
    model = AttentionModel()
    batch = batch_of(model, 256, 20, 64)
    for i in range(steps):
        loss = model.step(*batch, rate=20.0)
        if i % 10 == 0 or i + 1 == steps:
            print(f"step {i}: loss {loss.item():.4f}", flush=True)
    server = Server(model, 8, 20, bits=4)
    for i in range(20):
        p = server.next(batch[0][i * 8:i * 8 + 8])
    print(f"served {tuple(p.shape)}, mean probability {p.mean().item():.4f}", flush=True)


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 30)
