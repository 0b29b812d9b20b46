"""A small decoder trained on packed sequences, every step from the embedding
lookup to the clipped gradients through this package:

    python examples/train_block.py [--steps 60] [--dtype bf16|fp32]

    x = embedding(tokens)                                  lookup, padding skipped
    x, n = block_norm(x, w_pre)                            the first norm
    per layer, for attention and then for the MLP:
        b = attention(n W_qkv) W_o   or   gelu(n W_1) W_2  packed documents, shared key heads
        x, n = block_norm(x, b, w_post, gate, w_pre)       norm, gate, residual and the next norm in one
    loss = linear_cross_entropy(n, W, targets)             no logits in memory
    loss.backward(); clip_grad_norm(gradients); AdamW

The data are documents of random length in which each token follows from the
one before (t' = 5 t + 3 mod V) most of the time, so the loss falls quickly."""
import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_vocab_cross_gb300 as lce  # noqa: E402

PAD = 0
IGNORE = -100


class Decoder(torch.nn.Module):
    def __init__(self, vocab=1000, d=256, layers=2, heads=8, kv_heads=2, head_dim=32, dtype=torch.bfloat16):
        super().__init__()
        g = torch.Generator(device="cuda").manual_seed(0)
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim

        def mat(rows, cols):
            w = torch.randn(rows, cols, generator=g, device="cuda") * cols ** -0.5
            return torch.nn.Parameter(w.to(dtype))

        def vec(value):
            return torch.nn.Parameter(torch.full((d,), value, device="cuda", dtype=dtype))

        self.W = mat(vocab, d)            # shared by the lookup and the head
        self.first = vec(1.0)
        self.layers = torch.nn.ModuleList()
        for _ in range(layers):
            p = torch.nn.ParameterDict({
                "qkv": mat((heads + 2 * kv_heads) * head_dim, d), "o": mat(d, heads * head_dim),
                "up": mat(4 * d, d), "down": mat(d, 4 * d),
                "post1": vec(1.0), "gate1": vec(0.5), "pre1": vec(1.0),
                "post2": vec(1.0), "gate2": vec(0.5), "pre2": vec(1.0)})
            self.layers.append(p)

    def forward(self, tokens, cu, targets):
        x = lce.embedding(self.W, tokens, PAD)
        x, n = lce.block_norm(x, w_pre=self.first)
        for p in self.layers:
            qkv = (n @ p["qkv"].T).unflatten(1, (-1, self.head_dim))
            q, k, v = qkv.split([self.heads, self.kv_heads, self.kv_heads], 1)
            b = lce.attention(q, k, v, cu).flatten(1) @ p["o"].T
            x, n = lce.block_norm(x, b, w_post=p["post1"], gate=p["gate1"], w_pre=p["pre1"])
            b = F.gelu(n @ p["up"].T) @ p["down"].T
            x, n = lce.block_norm(x, b, w_post=p["post2"], gate=p["gate2"], w_pre=p["pre2"])
        return lce.linear_cross_entropy(n, self.W, targets, IGNORE)


def batch(g, vocab, tokens=2048):
    """Documents packed into one row, the row padded at its end."""
    lens = []
    while sum(lens) < tokens - 300:
        lens.append(int(torch.randint(20, 300, (1,), generator=g)))
    ids, targets = torch.full((tokens,), PAD), torch.full((tokens,), IGNORE)
    at = 0
    for n in lens:
        noise = (torch.rand(n + 1, generator=g) < 0.1).tolist()
        other = torch.randint(1, vocab, (n + 1,), generator=g).tolist()
        t = other[:1]
        for i in range(1, n + 1):
            t.append(other[i] if noise[i] else (5 * t[-1] + 3) % (vocab - 1) + 1)
        ids[at:at + n], targets[at:at + n] = torch.tensor(t[:-1]), torch.tensor(t[1:])
        at += n
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    return ids.cuda(), cu.cuda(), targets.cuda()


def train(steps=60, dtype=torch.bfloat16, max_norm=1.0, log=None):
    """Losses and gradient norms by step."""
    vocab = 1000
    model = Decoder(vocab, dtype=dtype)
    params = list(model.parameters())
    opt = torch.optim.AdamW(params, lr=2e-3, weight_decay=0.0)
    g = torch.Generator().manual_seed(1)
    batches = [batch(g, vocab) for _ in range(8)]
    losses, norms = [], []
    for step in range(steps):
        loss = model(*batches[step % len(batches)])
        opt.zero_grad(set_to_none=True)
        loss.backward()
        norm = lce.clip_grad_norm([p.grad for p in params], max_norm)
        opt.step()
        losses.append(loss.detach())
        norms.append(norm)
        if log and (step % 10 == 0 or step + 1 == steps):
            log(f"step {step:4d}  loss {loss.item():.4f}  gradient norm {norm.item():.3f}")
    return torch.stack(losses).tolist(), torch.stack(norms).tolist()


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--dtype", choices=["bf16", "fp32"], default="bf16")
    a = ap.parse_args()
    train(a.steps, torch.bfloat16 if a.dtype == "bf16" else torch.float32, log=print)
