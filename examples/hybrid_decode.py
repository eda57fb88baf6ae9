"""A small hybrid stack served through the library: gated-delta layers (pace_prefill_chunk,
pace_decode_step) and one attention layer (pace_rotary, pace_cache_write, pace_cache_attention).

    python examples/hybrid_decode.py

1. A prompt goes through all layers at once: the delta layers in chunked prefill, the attention
   layer as a chain of drafted tokens over an empty cache.
2. Tokens are decoded one by one: every layer's single-token form.
3. A tree of drafted tokens is put to the attention layer.  The cache holds the drafts behind the
   context; the best path is accepted, its keys and values are written again at their final
   positions, and the delta layers then take the accepted tokens.

Weights and inputs are random (there is no model here); what is checked is that the forms agree:
decoding token by token gives what one chunk gives, and every path of the tree what decoding that
path gives.  Prints the largest differences; main() returns them.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import bit_recurrent_state_amd as pace  # noqa: E402

B, WIDTH, HEADS, KV_HEADS, D, ROTARY, PAGE, MAX_PAGES = 2, 512, 8, 2, 128, 64, 64, 8
BF16 = torch.bfloat16


class DeltaLayer:
    """One gated-delta layer: packed state, decode buffer, random projections."""

    def __init__(self, gen):
        self.cfg = pace.pace4(B=B, Hv=HEADS, Hk=HEADS // 2, d=D)
        sizes = pace.layout(self.cfg)
        self.state = torch.zeros(sizes["state_bytes"], dtype=torch.uint8, device="cuda")
        self.buffer = torch.zeros(sizes["buffer_bytes"], dtype=torch.uint8, device="cuda")
        n = (HEADS // 2) * D
        self.w = weight(gen, WIDTH, 2 * n + HEADS * D + 2 * HEADS)
        self.out = weight(gen, HEADS * D, WIDTH)

    def inputs(self, x):
        n = (HEADS // 2) * D
        q, k, v, a, b = (x @ self.w).split([n, n, HEADS * D, HEADS, HEADS], dim=-1)
        unit = lambda t: torch.nn.functional.normalize(t.float().unflatten(-1, (-1, D)), dim=-1).to(BF16)  # noqa: E731
        decay = torch.exp(-torch.nn.functional.softplus(a.float() - 4)).contiguous()
        return unit(q), unit(k), v.unflatten(-1, (-1, D)).contiguous(), decay, torch.sigmoid(b.float()).contiguous()

    def prompt(self, x):
        q, k, v, a, b = self.inputs(x)
        o = torch.empty_like(v)
        pace.prefill_chunk(self.cfg, self.state, q, k, v, a, b, o)
        return x + o.flatten(-2) @ self.out

    def step(self, x):
        q, k, v, a, b = self.inputs(x)
        o = torch.empty_like(v)
        pace.decode_step(self.cfg, self.state, self.buffer, q, k, v, a, b, o)
        return x + o.flatten(-2) @ self.out


class AttentionLayer:
    """One attention layer over an 8-bit paged cache, half of every head rotated."""

    def __init__(self, gen):
        self.cfg = pace.CacheConfig(B=B, Hq=HEADS, Hkv=KV_HEADS, d=D, num_pages=B * MAX_PAGES, max_pages=MAX_PAGES,
                                    kind="int8", group=64, page=PAGE)
        self.rot = pace.RotaryConfig(Hq=HEADS, Hk=KV_HEADS, d=D, rd=ROTARY)
        self.cache = torch.zeros(pace.cache_layout(self.cfg)["cache_bytes"], dtype=torch.uint8, device="cuda")
        # pages are handed out in any order; here once, at random
        self.table = torch.randperm(B * MAX_PAGES, generator=gen, device="cuda").to(torch.int32).view(B, MAX_PAGES)
        freqs, self.magnitude = pace.rotary_freqs(ROTARY, 1e6)
        self.freqs = torch.from_numpy(freqs).cuda()
        self.w = weight(gen, WIDTH, (HEADS + 2 * KV_HEADS) * D)
        self.out = weight(gen, HEADS * D, WIDTH)

    def attend(self, x, lens, depth, slots, tree=None):
        """x [B, T, WIDTH]; lens [B] cached tokens; depth [T] a token's distance behind them (its
        position is lens + depth); slots [T] where its key and value are kept behind them."""
        T = x.shape[1]
        qkv = x @ self.w
        # slices of the projection go in as they are
        q, k, v = (t.unflatten(-1, (-1, D)) for t in qkv.split([HEADS * D, KV_HEADS * D, KV_HEADS * D], dim=-1))
        at = lambda d: (lens[:, None] + d[None, :]).to(torch.int32).contiguous()  # noqa: E731
        rows = lambda t: t.as_strided((B * T, *t.shape[2:]), (qkv.shape[-1], D, 1), t.storage_offset())  # noqa: E731
        pace.rotary(self.rot, at(depth).view(-1), self.freqs, rows(q), rows(k), rows(q), rows(k), magnitude=self.magnitude)
        pace.cache_write(self.cfg, self.cache, self.table, at(slots), k, v)
        o = torch.empty((B, T, HEADS, D), dtype=BF16, device="cuda")
        longest = MAX_PAGES * PAGE
        n = pace.cache_attention_workspace_bytes(self.cfg, T, longest)
        scratch = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
        pace.cache_attention(self.cfg, self.cache, self.table, q, lens, o, tree=tree, max_len=longest, workspace=scratch)
        return x + o.flatten(-2) @ self.out, k, v


def weight(gen, n, m):
    return (torch.randn((n, m), generator=gen, device="cuda") / n ** 0.5).to(BF16)


def off(a, b):
    return float((a.float() - b.float()).abs().max() / b.float().abs().max())


def main(prompt=150, steps=11):
    gen = torch.Generator(device="cuda").manual_seed(0)
    delta, attention = [DeltaLayer(gen) for _ in range(3)], AttentionLayer(gen)
    x = torch.randn((B, prompt + steps, WIDTH), generator=gen, device="cuda").to(BF16)
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    order = torch.arange(prompt + steps, device="cuda")

    # 1. the prompt
    y = x[:, :prompt]
    for layer in delta:
        y = layer.prompt(y)
    attention.attend(y, lens, order[:prompt], order[:prompt])
    lens += prompt

    # 2. token by token; the attention layer's inputs are kept to run them as one chunk as well
    inputs, outputs = [], []
    for t in range(prompt, prompt + steps):
        z = x[:, t]
        for layer in delta:
            z = layer.step(z)
        inputs.append(z)
        outputs.append(attention.attend(z[:, None], lens, order[:1], order[:1])[0][:, 0])
        lens += 1
    back = lens - steps
    chunk = attention.attend(torch.stack(inputs, 1), back, order[:steps], order[:steps])[0]
    found = {"token by token against one chunk": off(torch.stack(outputs, 1), chunk)}

    # 3. a tree of drafts behind the context: 0 -> (1 -> 3 -> 5, 2 -> 4)
    parents = [-1, 0, 0, 1, 2, 3]
    depth = torch.tensor([0, 1, 1, 2, 2, 3], device="cuda")
    drafts = torch.randn((B, len(parents), WIDTH), generator=gen, device="cuda").to(BF16)
    bits = torch.from_numpy(pace.tree_bits(parents))[None].cuda()
    checked, k, v = attention.attend(drafts, lens, depth, order[: len(parents)], tree=bits)
    for path in ([0, 2, 4], [0, 1, 3, 5]):
        for i, node in enumerate(path):                 # decode the path alone, over the drafts' places
            alone = attention.attend(drafts[:, node: node + 1], lens + i, order[:1], order[:1])[0]
            name = f"tree against path {path}"
            found[name] = max(found.get(name, 0.0), off(checked[:, node: node + 1], alone))
    # the longer path is accepted: its keys and values move to their final places, the others' are
    # left behind the new end, and the delta layers take its tokens
    final = torch.tensor([path.index(i) if i in path else -1 for i in range(len(parents))], device="cuda")
    at = torch.where(final >= 0, lens[:, None] + final, -1).to(torch.int32)
    pace.cache_write(attention.cfg, attention.cache, attention.table, at, k, v)
    for node in path:
        z = drafts[:, node]
        for layer in delta:
            z = layer.step(z)
    lens += len(path)
    torch.cuda.synchronize()
    for name, value in found.items():
        print(f"{name}: largest difference {value:.2e} of the largest value")
    return found


if __name__ == "__main__":
    main()
