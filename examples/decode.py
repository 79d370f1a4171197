"""A decoder of random weights that answers several questions about one text.

Each layer is the attention half (Q4_0 projections, a paged key/value cache, attention over the prompt and of single new
tokens) and the predictor-guided sparse FFN:

    h  = rms(x + W_o attention(W_qkv x))
    x' = rms(h + ffn(h))

The text goes through the prompt path into one slot of the cache.  That slot is forked once for every question, so all
questions share the text's whole pages, and each decoding step reads those once for the batch.  A step is captured into
a graph and replayed.  At the end half of the questions are released and the pool's pages are moved to its front.

    python examples/decode.py
    python examples/decode.py --width 8192 --heads 128 --kv-heads 8 --dim 64 --ffn 32768 --text 4096 --questions 32
"""
import argparse
import os
import sys
import time

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import activation_sparse_predict_amd as pi  # noqa: E402
import workload  # noqa: E402

ROWS = 32                                              # rows of one product or FFN call


def rms(v, eps=1e-5):
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + eps)


def q4_matrix(gen, rows, cols, batch):
    nibbles = torch.randint(0, 256, (rows, cols // 2), generator=gen, device=gen.device, dtype=torch.uint8)
    scales = (torch.rand(rows, cols // 32, generator=gen, device=gen.device) * (0.4 / cols ** 0.5)).to(torch.float16)
    return pi.Q4Matrix(nibbles, scales, batch=batch)


class Decoder:
    """Weights, cache and buffers of `slots` sequences."""

    def __init__(self, *, layers=2, width=4096, ffn=11008, rank=1024, heads=32, kv_heads=8, dim=128, page=16, pages=2048,
                 slots=33, max_pages=512, seed=1, device="cuda"):
        self.heads, self.kv_heads, self.dim, self.width, self.device = heads, kv_heads, dim, width, device
        gen = torch.Generator(device=device)
        gen.manual_seed(seed)
        cfg = workload.CONFIGS[1].with_(d=width, ffn=ffn, rank=rank, n_layers=layers)
        self.qkv = [q4_matrix(gen, (heads + 2 * kv_heads) * dim, width, ROWS) for _ in range(layers)]
        self.proj = [q4_matrix(gen, width, heads * dim, ROWS) for _ in range(layers)]
        self.ffn = [pi.DeviceLayer.upload(workload.make_layer(cfg, i), device) for i in range(layers)]
        self.ffn_ws = {}
        self.cache = pi.Cache.create(layers, pages, kv_heads, page, dim, slots, max_pages, device=device)
        self.one = torch.ones(slots, dtype=torch.int32, device=device)
        self.rows = torch.arange(slots + 1, dtype=torch.int32, device=device)
        self.prefix = torch.zeros(1, dtype=torch.int32, device=device)   # pages that all slots in use have in common
        self.used = set()                              # slots that were filled

    def ints(self, values):
        return torch.tensor(values, dtype=torch.int32, device=self.device)

    def _ffn(self, i, h):
        """rms(h + ffn(h)) of up to ROWS rows."""
        n = h.shape[0]
        if n not in self.ffn_ws:
            self.ffn_ws[n] = torch.empty(pi.workspace_bytes(self.ffn[i:i + 1], n), dtype=torch.uint8, device=self.device)
        out = torch.empty_like(h)
        pi.ffn_stack(self.ffn[i:i + 1], h, out, ws=self.ffn_ws[n], batch=n)
        return out

    def _layer(self, i, x, attend, trace):
        """One layer over rows x [n, width]; attend(qkv [n, heads + 2 kv_heads, dim], out [n, heads, dim])."""
        n = x.shape[0]
        qkv = torch.empty(n, self.heads + 2 * self.kv_heads, self.dim, dtype=torch.float16, device=self.device)
        out = torch.empty(n, self.heads, self.dim, dtype=torch.float16, device=self.device)
        y, nxt = torch.empty_like(x), torch.empty_like(x)
        for a in range(0, n, ROWS):
            pi.matvec(self.qkv[i], x[a:a + ROWS], qkv[a:a + ROWS].view(-1, self.qkv[i].rows))
        attend(qkv, out)
        for a in range(0, n, ROWS):
            pi.matvec(self.proj[i], out[a:a + ROWS].view(-1, self.heads * self.dim), y[a:a + ROWS])
        h = rms(x + y)
        for a in range(0, n, ROWS):
            nxt[a:a + ROWS] = self._ffn(i, h[a:a + ROWS].contiguous())
        if trace is not None:
            trace.append(dict(x=x, qkv=qkv, attn=out, y=y, h=h, out=nxt))
        return nxt

    def prompt(self, x, slot, trace=None):
        """Whole prompt x [tokens, width] into an empty slot; the outputs of its rows."""
        h, g = self.heads, self.kv_heads
        self.used.add(slot)
        self.prefix.zero_()
        cu, seqs = self.ints([0, x.shape[0]]), self.ints([slot])
        self.cache.extend(seqs, self.ints([x.shape[0]]))
        for i in range(len(self.ffn)):
            def attend(qkv, out):
                q, k, v = qkv[:, :h], qkv[:, h:h + g], qkv[:, h + g:]
                self.cache.append(i, k, v, cu, seqs)
                pi.attn_prompt(q, k, v, out, cu)
            x = self._layer(i, x, attend, trace)
        return x

    def step(self, x, seqs, trace=None):
        """One new token x [n, width] for each of the slots seqs; the outputs."""
        h, g, n = self.heads, self.kv_heads, x.shape[0]
        self.cache.extend(seqs, self.one[:n])
        for i in range(len(self.ffn)):
            def attend(qkv, out):
                self.cache.append(i, qkv[:, h:h + g], qkv[:, h + g:], self.rows[:n + 1], seqs)
                pi.attn_decode(self.cache, i, qkv[:, :h], out, prefix=self.prefix, seqs=seqs)
            x = self._layer(i, x, attend, trace)
        return x

    def share(self, parent, children, tokens):
        """Children continue the parent's `tokens` tokens; their common pages are read once from now on, unless slots are in use
        that hold something else."""
        self.cache.fork(self.ints([parent] * len(children)), self.ints(children))
        alone = self.used <= {parent, *children}
        self.prefix.fill_(tokens // self.cache.page if alone else 0)
        self.used.update(children)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("layers", 2), ("width", 4096), ("ffn", 11008), ("rank", 1024), ("heads", 32), ("kv-heads", 8),
                        ("dim", 128), ("page", 16), ("text", 1000), ("questions", 8), ("tokens", 64)):
        ap.add_argument("--" + name, type=int, default=value)
    a = ap.parse_args()
    per = (a.text + a.tokens + 8) // a.page + 2        # pages of one sequence
    pages = a.text // a.page + 1 + (a.questions + 1) * (a.tokens // a.page + 3)
    d = Decoder(layers=a.layers, width=a.width, ffn=a.ffn, rank=a.rank, heads=a.heads, kv_heads=a.kv_heads, dim=a.dim,
                page=a.page, pages=pages, slots=a.questions + 1, max_pages=per)
    gen = torch.Generator(device=d.device)
    gen.manual_seed(2)
    text = torch.randn(a.text, a.width, generator=gen, device=d.device)
    torch.cuda.synchronize()
    t = time.perf_counter()
    d.prompt(text, 0)
    torch.cuda.synchronize()
    print(f"text of {a.text} tokens: {(time.perf_counter() - t) * 1e3:.1f} ms", flush=True)

    slots = list(range(1, a.questions + 1))
    d.share(0, slots, a.text)
    seqs = d.ints(slots)
    x = torch.randn(a.questions, a.width, generator=gen, device=d.device)
    x.copy_(d.step(x, seqs))                           # once before the capture: workspaces are taken here
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        x.copy_(d.step(x, seqs))
    graph.replay()
    torch.cuda.synchronize()
    t, n = time.perf_counter(), max(1, a.tokens - 2)
    for _ in range(n):
        graph.replay()
    torch.cuda.synchronize()
    t = time.perf_counter() - t
    print(f"{a.questions} answers of {n} tokens: {t / n * 1e3:.3f} ms a step, {a.questions * n / t:.0f} tokens/s, "
          f"pages free {int(d.cache.words[0])} of {pages}", flush=True)

    d.cache.release(d.ints(slots[::2]))
    d.cache.compact()
    x.copy_(d.step(x, seqs)) if a.questions == 1 else d.step(x[1::2].contiguous(), d.ints(slots[1::2]))
    errors = d.cache.errors()
    print(f"half of them released, {int(d.cache.words[2])} pages in use moved to the front; error word {errors}", flush=True)
    if errors or not torch.isfinite(x).all():
        sys.exit(1)


if __name__ == "__main__":
    main()
