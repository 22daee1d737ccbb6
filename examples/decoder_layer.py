"""The first half of a decoder layer made of BitLinears, for serving and for training.

    python examples/decoder_layer.py            # one MI355X

Serving (AttentionBlock): several sequences share a prompt's beginning (a system
prompt), whose keys and values are held once.  A step takes the new tokens of every
sequence (whole prompts, or one token each) through
    norm of hidden + residual to int8 rows -> q, k, v BitLinears on those rows
    -> k, v to the int8 cache -> attention over the shared prefix and the sequence's
    own keys -> output BitLinear, whose result the next norm adds to the residual.
No position is encoded; a program that rotates q and k does it between the BitLinears
and the cache.

Training (NormedBitLinear): a BitLinear behind its norm.  The forward keeps the sum
and the int8 rows; the backward takes the BitLinear's straight-through input
gradient through the norm and adds the residual stream's.
"""
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from ternary_weight_linear_forward_amd import bitlinear as bl  # noqa: E402


class Linear:
    """Packed ternary weights [N x K] of one BitLinear."""

    def __init__(self, W):
        self.N, self.K = W.shape
        T, self.gamma = bl.quantize_weights(W)
        self.P = bl.pack(T)

    def __call__(self, Xq, beta, y_dtype=torch.bfloat16):
        return bl.forward(self.P, bl.LAYOUT_I2, self.gamma, Xq, self.N, self.K, beta=beta, y_dtype=y_dtype)


class AttentionBlock:
    """Norm, q / k / v, cache, attention and output of one layer, for up to 'seqs' sequences of at most 'max_own'
    tokens of their own behind a prefix of at most 'max_prefix'."""

    def __init__(self, wq, wk, wv, wo, norm, heads, kv_heads, seqs, max_own, max_prefix, page_tokens=64):
        self.q, self.k, self.v, self.o = (Linear(w) for w in (wq, wk, wv, wo))
        self.norm, self.heads, self.kv_heads, self.page = norm, heads, kv_heads, page_tokens
        self.D, self.max_own, self.max_prefix = wq.shape[0] // heads, max_own, max_prefix
        need = lambda n: (n + page_tokens - 1) // page_tokens  # noqa: E731
        dev = norm.device
        self.cache = bl.KVCache.empty(need(max_prefix) + seqs * need(max_own), kv_heads, self.D, page_tokens, dev)
        self.prefix_pages = torch.arange(need(max_prefix), dtype=torch.int32, device=dev)
        self.own_pages = (need(max_prefix) + torch.arange(seqs * need(max_own), dtype=torch.int32, device=dev)
                          ).reshape(seqs, need(max_own))
        self.own_len = torch.zeros(seqs, dtype=torch.int32, device=dev)
        self.held = [0] * seqs  # own_len as the host knows it
        self.prefix_len = 0

    def _slots(self, pages, positions):
        """Cache places of token positions of page lists [n, pages]."""
        page = pages.gather(1, (positions // self.page)[:, None]).squeeze(1)
        return page.long() * self.page + positions % self.page

    def _attend(self, hidden, residual, slots, own_pages, own_len, max_own, prefix_len, q_start, max_q):
        n = hidden.shape[0]
        h, xq, beta = bl.norm_quantize(hidden, self.norm, residual=residual)
        q, k, v = self.q(xq, beta), self.k(xq, beta), self.v(xq, beta)
        bl.cache_write(self.cache, k.view(n, self.kv_heads, self.D), v.view(n, self.kv_heads, self.D), slots)
        a = bl.attention(self.cache, q.view(n, self.heads, self.D), own_pages, own_len, max_own,
                         prefix_pages=self.prefix_pages, prefix_len=prefix_len, q_start=q_start, max_q=max_q)
        aq, abeta = bl.quantize_act(a.view(n, -1))
        return self.o(aq, abeta), h

    def load_prefix(self, hidden, residual):
        """The shared beginning, once: its tokens see one another and go to the prefix's pages."""
        n = hidden.shape[0]
        if n > self.max_prefix:
            raise ValueError(f"a prefix of {n} tokens in a block for {self.max_prefix}")
        at = torch.arange(n, device=hidden.device)
        pages = self.prefix_pages[None]
        out = self._attend(hidden, residual, self._slots(pages.expand(n, -1), at), pages,
                           torch.tensor([n], dtype=torch.int32, device=hidden.device), n, 0, None, n)
        self.prefix_len = n
        return out

    def step(self, hidden, residual, counts):
        """New tokens of every sequence, 'counts' of them each (hidden and residual hold them one sequence after
        the other): (the block's output, the sum that its norm kept) for the rest of the layer."""
        held = [n + c for n, c in zip(self.held, counts)]
        if len(counts) != len(self.held) or min(counts) < 0 or sum(counts) != hidden.shape[0] or max(held) > self.max_own:
            raise ValueError(f"{hidden.shape[0]} new tokens, counts {counts}: {len(self.held)} sequences hold "
                             f"{self.held} of {self.max_own}")
        self.held = held
        dev = hidden.device
        count = torch.tensor(counts, dtype=torch.int32, device=dev)
        start = torch.zeros(len(counts) + 1, dtype=torch.int32, device=dev)
        start[1:] = count.cumsum(0)
        seq = torch.repeat_interleave(torch.arange(len(counts), device=dev), count.long(), output_size=hidden.shape[0])
        at = torch.arange(hidden.shape[0], device=dev) - start[seq].long() + self.own_len[seq].long()
        self.own_len += count
        one = all(c == 1 for c in counts)
        return self._attend(hidden, residual, self._slots(self.own_pages[seq], at), self.own_pages, self.own_len,
                            self.max_own, self.prefix_len, None if one else start, max(counts))


class NormedBitLinear:
    """y = BitLinear(norm(x + residual)) with its gradients, for training with latent fp32 weights."""

    def __init__(self, W, norm):
        self.W, self.norm = W, norm

    def forward(self, x, residual=None):
        self.lin = Linear(self.W)  # (the latent weights change between steps)
        self.h, self.xq, self.beta = bl.norm_quantize(x, self.norm, residual=residual)
        return self.lin(self.xq, self.beta, torch.float32), self.h

    def backward(self, dY, dH=None):
        """(d x = d residual, d W, d norm) from the gradients of y and of the kept sum."""
        dN = bl.backward_dx(self.lin.P, bl.LAYOUT_I2, self.lin.gamma, dY, self.lin.K)
        dW = bl.backward_dw(self.xq, self.beta, dY, self.lin.K)
        dX, dnorm = bl.norm_backward(dN, self.h, self.norm, dH=dH)
        return dX, dW, dnorm


def random_block(width, heads, kv_heads, seqs, max_own, max_prefix, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    w = lambda n, k: torch.randn(n, k, generator=g, device=device) * k ** -0.5  # noqa: E731
    kv = width // heads * kv_heads
    return AttentionBlock(w(width, width), w(kv, width), w(kv, width), w(width, width),
                          1.0 + 0.1 * torch.randn(width, generator=g, device=device), heads, kv_heads, seqs, max_own,
                          max_prefix)


def main():
    width, heads, seqs, prefix, prompt, steps = 3200, 32, 16, 1000, 40, 50
    block = random_block(width, heads, heads, seqs, prompt + steps + 3, prefix)
    new = lambda n: torch.randn(n, width, device="cuda").bfloat16()  # noqa: E731
    block.load_prefix(new(prefix), new(prefix))
    block.step(new(seqs * prompt), new(seqs * prompt), [prompt] * seqs)
    x, r, ones = new(seqs), new(seqs), [1] * seqs
    for _ in range(3):
        block.step(x, r, ones)
    torch.cuda.synchronize()
    t = time.perf_counter()
    for _ in range(steps):
        block.step(x, r, ones)
    torch.cuda.synchronize()
    t = (time.perf_counter() - t) / steps
    print(f"decode: width {width}, {heads} heads, {seqs} sequences behind {prefix} shared tokens: "
          f"{t * 1e6:.0f} us a step of this half of a layer, {seqs / t:.0f} tokens/s")
    lin = NormedBitLinear(torch.randn(width, width, device="cuda") * width ** -0.5, torch.ones(width, device="cuda"))
    y, _ = lin.forward(new(512), new(512))
    dx, dw, dn = lin.backward(torch.randn_like(y) * 0.01)
    print(f"training: d x {tuple(dx.shape)} {dx.dtype}, d W {tuple(dw.shape)}, d norm {tuple(dn.shape)}")


if __name__ == "__main__":
    main()
