"""A hybrid decoder stack served step by step: three KDA layers to one softmax
attention layer, the layout of page "Kimi K3：架构、训练与百万 Token Agentic RL 技术解读" §2,
with random weights (no projections or norms of a trained model exist here).

One ``step`` takes any mix of requests, new prompts beside running ones:

* ``kda_page_map`` turns the requests' lengths into the packed sequences' offsets
  (what ``kda_chunk_fwd`` takes), the new tokens' slots in the attention layer's
  4-bit cache and its block tables;
* a KDA layer runs ``kda_chunk_fwd`` over the packed tokens from each request's
  recurrent state, or ``kda_decode_step`` when every request has one new token;
* the attention layer writes the new keys and values (``kda_kv4_append``) and
  attends over what is cached (``kda_kv4_attention``).

Run it on a GPU: ``python examples/hybrid_decoder.py [requests] [prompt] [steps]``.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import linear_attention_recurrence_chunk_gb300 as kda  # noqa: E402

D = 128   # head size


def _norm(x):
    return x * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6).to(x.dtype)


def _unit(x):
    return (x.float() / x.float().norm(dim=-1, keepdim=True).clamp(min=1e-6)).to(x.dtype)


class HybridDecoder:
    """``blocks`` x (three KDA layers, one attention layer) over ``requests`` requests
    of at most ``max_len`` tokens each."""

    def __init__(self, requests, max_len, blocks=1, hidden=512, heads=4, q_heads=8, kv_heads=2, page_size=64, seed=0):
        self.n, self.heads, self.q_heads, self.kv_heads, self.page = requests, heads, q_heads, kv_heads, page_size
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(a, b):
            return (torch.randn(a, b, device="cuda", generator=g) * a ** -0.5).to(torch.bfloat16)

        self.layers = []
        row = -(-max_len // page_size)
        pages = requests * row
        for i in range(4 * blocks):
            if i % 4 < 3:   # KDA: q, k, v, g, beta projections and the recurrent states
                self.layers.append({"in": weight(hidden, 4 * heads * D + heads), "out": weight(heads * D, hidden),
                                    "state": torch.zeros(requests, heads, D, D, device="cuda")})
            else:           # attention: q, k, v projections and the cache
                self.layers.append({"in": weight(hidden, (q_heads + 2 * kv_heads) * D), "out": weight(q_heads * D, hidden),
                                    "cache": kda.kda_kv4_cache(pages, kv_heads, page_size, D)})
        # the attention layers share the block tables: a page has the same number in each layer's cache
        self.table = torch.full((requests, row), -1, dtype=torch.int32, device="cuda")
        self.free = torch.randperm(pages, device="cuda", generator=g).int()
        self.next_free = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(requests, dtype=torch.int32, device="cuda")

    def step(self, x, new_lens):
        """x: bf16 [tokens, hidden], the requests' new tokens packed in order; new_lens:
        how many each request has (host list).  Returns the stack's output for them."""
        T, most = x.shape[0], max(new_lens)
        new = torch.tensor(new_lens, dtype=torch.int32, device="cuda")
        cu, total, slots, _, self.next_free = kda.kda_page_map(self.lens, new, self.table, self.free, self.next_free, self.page, T)
        single = min(new_lens) == most == 1
        for layer in self.layers:
            p = _norm(x) @ layer["in"]
            if "state" in layer:
                w = self.heads * D
                q, k, v, g = (p[:, i * w:(i + 1) * w].reshape(T, self.heads, D) for i in range(4))
                beta = torch.sigmoid(p[:, 4 * w:].float())
                q, k, v, g = _unit(q), _unit(k), v.contiguous(), g.contiguous()
                if single:
                    o = kda.kda_decode_step(q, k, v, g, beta, layer["state"])
                else:
                    o, _ = kda.kda_chunk_fwd(q[None], k[None], v[None], g[None], beta[None], initial_state=layer["state"],
                                             cu_seqlens=cu, final_state=layer["state"])
                    o = o[0]
            else:
                a, b = self.q_heads * D, (self.q_heads + self.kv_heads) * D
                q, k, v = (y.view(T, -1, D) for y in (p[:, :a], p[:, a:b], p[:, b:]))   # parts of the projection as they lie
                kda.kda_kv4_append(k, v, slots, layer["cache"])
                o = kda.kda_kv4_attention(q, layer["cache"], self.table, total, cu_seqlens=cu, max_q_len=most)
            x = x + o.reshape(T, -1) @ layer["out"]
        self.lens = total
        return x


def main(requests=8, prompt=1000, steps=32):
    gen = torch.Generator(device="cuda").manual_seed(1)
    model = HybridDecoder(requests, prompt + steps + 2)
    lens = [max(1, prompt * (i + 1) // requests) for i in range(requests)]
    y = model.step(torch.randn(sum(lens), 512, device="cuda", generator=gen).bfloat16(), lens)
    last = torch.tensor(lens, device="cuda").cumsum(0) - 1
    x = y[last]
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    for i in range(steps + 2):
        if i == 2:   # two steps to warm up
            start.record()
        x = _norm(model.step(x, [1] * requests))   # (a real decoder would sample a token and embed it)
    end.record()
    torch.cuda.synchronize()
    status, code = kda.kda_device_error()
    assert status == 0, (status, code)
    print(f"{requests} requests, prompts up to {prompt} tokens: {steps} decode steps of 4 layers, "
          f"{start.elapsed_time(end) / steps * 1e3:.0f} us a step; {int(model.next_free)} of {model.free.numel()} pages in use")
    return x


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:]))
