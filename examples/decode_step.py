"""One sparse-attention decode step through the library: append the new tokens to
the latent cache, select the top-k of each request's scores, attend over the
selection.

    python examples/decode_step.py [requests] [context]

Scores are random here (a model's indexer writes them); sizes are those of the
library's benchmark: 64-token pages, k = 2048, a 512-value latent, 16 heads.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import exact_bf16_top_gb300 as tk  # noqa: E402

PAGE, K, HEADS, LATENT, ROPE = 64, 2048, 16, 512, 64


def make(requests: int, context: int, seed: int = 0) -> dict:
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)

    pages = -(-context // PAGE)
    lens = torch.randint(max(1, context // 2), context + 1, (requests,), generator=g, device="cuda").int()
    table = torch.randperm(requests * pages, generator=g, device="cuda").view(requests, pages).int()
    last = (lens - 1).long()                       # the new token's position
    slots = (table.gather(1, (last // PAGE)[:, None])[:, 0] * PAGE + last % PAGE).int()
    angle = (torch.arange(context, device="cuda", dtype=torch.float64)[:, None]
             * 10000.0 ** (-torch.arange(0, ROPE, 2, device="cuda", dtype=torch.float64) / ROPE))
    return dict(cache=normal(requests * pages * PAGE, LATENT + ROPE), lens=lens, table=table, slots=slots,
                cos_sin=torch.cat((angle.cos(), angle.sin()), 1).float(), weight=1 + normal(LATENT) / 8,
                latent=normal(requests, LATENT), key_rope=normal(requests, ROPE),
                query_rope=normal(requests, HEADS, ROPE), query=normal(requests, HEADS, LATENT + ROPE),
                scores=normal(requests, -(-context // 8) * 8), scale=192 ** -0.5)


def step(s: dict):
    """(attention output, log-sum-exp, selected rows) of every request's new token."""
    tk.latent_append(s["cache"], s["latent"], s["key_rope"], s["lens"] - 1, s["cos_sin"], s["slots"],
                     weight=s["weight"], query_rope=s["query_rope"], query=s["query"])
    rows = tk.select(s["scores"], s["lens"], K, tk.TOKEN, s["table"], PAGE)
    out, lse = tk.latent_attend_selected(s["query"], s["cache"], rows, s["scale"], latent=LATENT, lse=True)
    return out, lse, rows


def main():
    requests = int(sys.argv[1]) if len(sys.argv) > 1 else 32
    context = int(sys.argv[2]) if len(sys.argv) > 2 else 16384
    s = make(requests, context)
    out, lse, rows = step(s)
    whole, whole_lse = tk.latent_attend_paged(s["query"], s["cache"], s["lens"], s["table"], s["scale"],
                                              page_size=PAGE, latent=LATENT, lse=True)
    torch.cuda.synchronize()
    share = torch.exp(lse - whole_lse).mean().item()
    print(f"{requests} requests: {tuple(out.shape)} from {(rows >= 0).sum().item()} selected rows, "
          f"{share:.3f} of the softmax of all {int(s['lens'].sum())} tokens")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(s)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    graph.replay()
    start.record()
    for _ in range(20):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"a step (append, select, attend) in a graph: {start.elapsed_time(end) * 50:.1f} us")


if __name__ == "__main__":
    main()
