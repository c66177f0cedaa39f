"""A small hybrid language model served token by token: three KDA layers to one layer of full attention.

    python examples/serve_hybrid.py [--layers 4] [--batch 4] [--prompt 200] [--tokens 32] [--no-graph]

The weights are random (no checkpoint is involved); what the example shows is the path of a prompt and of the tokens
after it:

* the prompts, of different lengths, are packed: KDA layers take them in chunks (``chunk_fwd`` with ``cu_seqlens``), and
  its final states go to the slots of the batch; attention layers append all rows to the paged cache at once
  (``cache_append``) and attend row by row (``cache_attend``, each prompt row a sequence of its own over its pages);
* every token after them is one ``step`` per KDA layer and one ``cache_append`` + ``cache_attend`` per attention layer,
  captured once in a CUDA graph and replayed.

At the end the whole sequences are run once more as prompts: their logits have to be those of the decoding.
"""
from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import chunked_gated_delta_10_gb300 as kda  # noqa: E402

DIM, HEADS, QUERY, CACHE, D, VOCAB, PAGE = 256, 2, 4, 2, 128, 1000, 16


def norm(x):
    return torch.nn.functional.rms_norm(x.float(), x.shape[-1:]).to(x.dtype)


def rope_table(positions, device):
    rate = 10000.0 ** (-torch.arange(0, D, 2, device=device, dtype=torch.float64) / D)
    angle = torch.arange(positions, device=device, dtype=torch.float64)[:, None] * rate
    return torch.cat([angle.cos(), angle.sin()], 1).float()


class KdaLayer:
    """q, k (normalised), v, the gate and beta from one projection; the state of sequence n in slot n."""

    def __init__(self, rand, batch, **_):
        self.sizes = [HEADS * D, HEADS * D, HEADS * D, HEADS * D, HEADS]
        self.into, self.out = rand(DIM, sum(self.sizes)), rand(HEADS * D, DIM)
        self.state = torch.zeros(batch, HEADS, D, D, device="cuda")
        self.slots = torch.arange(batch, dtype=torch.int32, device="cuda")

    def inputs(self, x):  # x [N, T, DIM]
        q, k, v, g, b = (x @ self.into).split(self.sizes, -1)
        heads = lambda t: t.unflatten(-1, (HEADS, D))  # noqa: E731
        unit = lambda t: torch.nn.functional.normalize(heads(t).float(), dim=-1).to(x.dtype)  # noqa: E731
        gate = torch.nn.functional.logsigmoid(heads(g).float() + 3)
        return [t.contiguous() for t in (unit(q), unit(k), heads(v), gate, torch.sigmoid(b.float()).to(x.dtype))]

    def prompt(self, x, batch):
        o, state, _ = kda.chunk_fwd(*self.inputs(x[None]), cu_seqlens=batch["cu_host"])
        self.state.copy_(state)
        return o[0].flatten(1) @ self.out

    def token(self, x, batch):
        o = kda.step(*self.inputs(x[:, None]), self.state, slots=self.slots)
        return o.flatten(1) @ self.out


class AttentionLayer:
    """Grouped queries over a paged cache, positions by rotation."""

    def __init__(self, rand, batch, pages, **_):
        self.sizes = [QUERY * D, CACHE * D, CACHE * D]
        self.into, self.out = rand(DIM, sum(self.sizes)), rand(QUERY * D, DIM)
        self.cache = kda.new_cache(pages, PAGE, CACHE, D, D)

    def inputs(self, x):  # rows of one projection: the heads of a row are contiguous, the rows lie apart
        return [t.unflatten(-1, (n, D)) for t, n in zip((x @ self.into).split(self.sizes, -1), (QUERY, CACHE, CACHE))]

    def prompt(self, x, batch):
        q, k, v = self.inputs(x)
        q = kda.cache_append(k, v, *self.cache, batch["table"], torch.zeros_like(batch["lens"]), q=q, rope=batch["rope"],
                             cu_seqlens=batch["cu"], status=batch["status"])
        o, _ = kda.cache_attend(q, *self.cache, batch["row_table"], batch["row_lens"], status=batch["status"])
        return o.flatten(1) @ self.out

    def token(self, x, batch):
        q, k, v = self.inputs(x)
        q = kda.cache_append(k, v, *self.cache, batch["table"], batch["lens"], q=q, rope=batch["rope"],
                             status=batch["status"])
        o, _ = kda.cache_attend(q, *self.cache, batch["table"], batch["lens"] + 1, status=batch["status"])
        return o.flatten(1) @ self.out


class Model:
    def __init__(self, layers, batch, longest, seed=0):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rand = lambda a, b: (torch.randn(a, b, generator=gen, device="cuda") / a ** 0.5).bfloat16()  # noqa: E731
        width = -(-longest // PAGE)
        self.embed = rand(VOCAB, DIM) * VOCAB ** 0.5
        self.layers = [(AttentionLayer if i % 4 == 3 else KdaLayer)(rand, batch=batch, pages=batch * width)
                       for i in range(layers)]
        table = torch.randperm(batch * width, generator=gen, device="cuda").to(torch.int32).view(batch, width)
        self.batch = dict(table=table, lens=torch.zeros(batch, dtype=torch.int32, device="cuda"),
                          rope=rope_table(longest, "cuda"), status=torch.zeros(1, dtype=torch.int32, device="cuda"))

    def run(self, tokens, how):
        x = self.embed[tokens]
        for layer in self.layers:
            x = x + getattr(layer, how)(norm(x), self.batch)
        return norm(x).float() @ self.embed.float().T

    def prompts(self, prompts):
        """Logits of every row of the packed prompts."""
        b, lens = self.batch, torch.tensor([len(p) for p in prompts])
        b["cu_host"] = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)])
        b["cu"] = b["cu_host"].cuda()
        of = torch.repeat_interleave(torch.arange(len(prompts)), lens).cuda()
        b["row_table"] = b["table"][of]
        b["row_lens"] = torch.cat([torch.arange(1, n + 1) for n in lens.tolist()]).to(torch.int32).cuda()
        logits = self.run(torch.cat(prompts).cuda(), "prompt")
        b["lens"].copy_(lens)
        return logits

    def token(self, tokens):
        """Logits of one more token of every sequence."""
        logits = self.run(tokens, "token")
        self.batch["lens"].add_(1)
        return logits


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--layers", type=int, default=4)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--prompt", type=int, default=200, help="longest prompt")
    ap.add_argument("--tokens", type=int, default=32)
    ap.add_argument("--no-graph", action="store_true")
    a = ap.parse_args(argv)
    kda.build()
    gen = torch.Generator().manual_seed(1)
    lens = torch.randint(1, a.prompt + 1, (a.batch,), generator=gen).tolist()
    prompts = [torch.randint(0, VOCAB, (n,), generator=gen) for n in lens]
    model = Model(a.layers, a.batch, a.prompt + a.tokens)

    ends = torch.tensor(lens).cumsum(0) - 1
    logits = model.prompts(prompts)[ends.cuda()]
    seen, said = [logits], [logits.argmax(-1)]
    token = said[0].clone()
    step = model.token
    if not a.no_graph:
        saved = [x.clone() for x in (model.batch["lens"], *(y.state for y in model.layers if isinstance(y, KdaLayer)))]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            model.token(token)  # a first run outside of the capture
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = model.token(token)
        for x, y in zip((model.batch["lens"], *(y.state for y in model.layers if isinstance(y, KdaLayer))), saved):
            x.copy_(y)

        def step(_):
            graph.replay()
            return out

    torch.cuda.synchronize()
    began = time.perf_counter()
    for _ in range(a.tokens - 1):
        logits = step(token)
        token.copy_(logits.argmax(-1))
        seen.append(logits.clone())
        said.append(token.clone())
    torch.cuda.synchronize()
    spent = time.perf_counter() - began
    if a.tokens > 1:
        print(f"{a.batch} sequences, {a.tokens - 1} tokens each after the first: {spent / (a.tokens - 1) * 1e6:.0f} us a token")

    # the same sequences once more, as prompts: row lens[n] - 1 + i of sequence n predicted its token i
    whole = [torch.cat([p, torch.stack(said, 1)[n, :-1].cpu()]) for n, p in enumerate(prompts)]
    again = model.prompts(whole)
    starts = torch.tensor([0] + [len(w) for w in whole]).cumsum(0)[:-1] + torch.tensor(lens) - 1
    rows = starts[:, None] + torch.arange(a.tokens)
    again = again[rows.cuda()]
    err = float((again - torch.stack(seen, 1)).norm() / again.norm())
    same = float((again.argmax(-1) == torch.stack(said, 1)).float().mean())
    print(f"decoding against the same sequences as prompts: logits differ by {err:.2e} (relative L2), {same:.1%} of tokens equal")
    if int(model.batch["status"]):
        raise SystemExit("a page or a position did not exist")
    return err


if __name__ == "__main__":
    if main() > 0.05:
        raise SystemExit("the decoding is not the prompt's")
