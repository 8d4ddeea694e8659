"""A small language model on linear attention, trained and served.

    python examples/recall.py [--steps N]

Documents are a block of distinct random tokens, twice over; the model learns
to recall what followed a token the first time.  Keys come from the token
before, so that the state maps each token to its successor.  Training runs
`linattn` and `linattn_grad` over packed documents of unequal length, whose
ends `runs_layout_u32` lays out; serving reads the prompts with one `linattn`,
then writes a token at a time with `linattn_step` and `sample_logits`.
"""
import argparse
import math
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import prefix_scan_amd as ps  # noqa: E402


class LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay, scale, ends):
        ctx.save_for_backward(q, k, v, log_decay, ends)
        ctx.scale = scale
        return ps.linattn(q, k, v, log_decay, scale, ends)[0]

    @staticmethod
    def backward(ctx, dout):
        q, k, v, log_decay, ends = ctx.saved_tensors
        dq, dk, dv, _ = ps.linattn_grad(dout.contiguous(), q, k, v, log_decay, ctx.scale, ends)
        return dq, dk, dv, None, None, None


class Recall(torch.nn.Module):
    def __init__(self, vocab=64, width=128, heads=4, head_width=64):
        super().__init__()
        self.vocab, self.heads, self.head_width = vocab, heads, head_width
        self.scale = 1.0 / math.sqrt(head_width)
        self.embed = torch.nn.Embedding(vocab + 1, width)      # the last: before a document
        self.q, self.k, self.v = (torch.nn.Linear(width, heads * head_width, bias=False) for _ in range(3))
        self.head = torch.nn.Linear(heads * head_width, vocab, bias=False)
        # From no decay to a memory of 32 tokens.
        decay = torch.tensor([0.0] + [math.log1p(-2.0 ** -(9 - h)) for h in range(1, heads)])
        self.register_buffer("log_decay", decay)

    def rows(self, tokens, before):
        """bf16 rows [N, H, D] of q, k and v."""
        x, y = self.embed(tokens), self.embed(before)
        cut = lambda t: t.view(-1, self.heads, self.head_width).bfloat16()  # noqa: E731
        return cut(self.q(x)), cut(self.k(y)), cut(self.v(x))

    def logits(self, out):
        return self.head(out.flatten(1).float())

    def forward(self, tokens, before, ends):
        return self.logits(LinearAttention.apply(*self.rows(tokens, before), self.log_decay, self.scale, ends))


def documents(count, vocab, longest, gen):
    """Packed tokens, the token before each, and the documents' lengths."""
    lens = torch.randint(4, longest + 1, (count,), generator=gen)
    docs = [torch.randperm(vocab, generator=gen)[:n].repeat(2) for n in lens.tolist()]
    before = [F.pad(d[:-1], (1, 0), value=vocab) for d in docs]
    return torch.cat(docs).cuda(), torch.cat(before).cuda(), (2 * lens).to(torch.int32).cuda()


def train(model, steps, count=32, longest=40, seed=0):
    """Losses of the tokens that can be recalled, a step each."""
    gen = torch.Generator().manual_seed(seed)
    adam = torch.optim.Adam(model.parameters(), lr=3e-3)
    losses = []
    for _ in range(steps):
        tokens, before, lens = documents(count, model.vocab, longest, gen)
        ends, _ = ps.runs_layout_u32(lens, want_entries=False)
        logits = model(tokens, before, ends)
        # From the second block on, but for each document's last token.
        doc = torch.repeat_interleave(torch.arange(count, device="cuda"), lens.long())
        at = torch.arange(len(tokens), device="cuda") - (ends - lens)[doc]
        known = (at >= lens[doc] // 2) & (at + 1 < lens[doc])
        loss = F.cross_entropy(logits[known], torch.roll(tokens, -1)[known])
        adam.zero_grad()
        loss.backward()
        adam.step()
        losses.append(loss.detach())
    return [float(x) for x in losses]


@torch.no_grad()
def serve(model, prompts, new, u, temperature=1.0, top_k=0, top_p=1.0):
    """`new` tokens after each prompt (lists of tokens) by the random numbers
    u [new, prompts]: (tokens [new, prompts], the states after the last)."""
    lens = torch.tensor([len(p) for p in prompts], dtype=torch.int32, device="cuda")
    ends, _ = ps.runs_layout_u32(lens, want_entries=False)
    tokens = torch.tensor(sum(prompts, []), device="cuda")
    before = torch.tensor(sum(([model.vocab] + p[:-1] for p in prompts), []), device="cuda")
    out, state = ps.linattn(*model.rows(tokens, before), model.log_decay, model.scale, ends, want_state=True)
    last = ends.long() - 1
    out, token = out[last], tokens[last]
    written = []
    for i in range(new):
        following = ps.sample_logits(model.logits(out), u[i], temperature, top_k, top_p)[0].long()
        written.append(following)
        out, state = ps.linattn_step(*model.rows(following, token), model.log_decay, state, model.scale)
        token = following
    return torch.stack(written), state


def main():
    parser = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    parser.add_argument("--steps", type=int, default=200)
    args = parser.parse_args()
    torch.manual_seed(0)
    model = Recall().cuda()
    losses = train(model, args.steps)
    print("loss %.3f -> %.3f over %d steps" % (losses[0], losses[-1], len(losses)))
    gen = torch.Generator().manual_seed(1)
    blocks = [torch.randperm(model.vocab, generator=gen)[:n].tolist() for n in (8, 13, 30)]
    new = 8
    u = torch.rand((new, len(blocks)), generator=gen).cuda()
    written, _ = serve(model, [b + b[:1] for b in blocks], new, u, temperature=0.7, top_k=20, top_p=0.9)
    for block, row in zip(blocks, written.t().tolist()):
        want = (block * 2)[1:new + 1]
        print("after %s ... wrote %s, %d of %d recalled" % (
            block[:4], row, sum(a == b for a, b in zip(row, want)), new))


if __name__ == "__main__":
    main()
