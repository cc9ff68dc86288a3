"""Greedy decoding with a tree of drafted tokens, on a small synthetic model of
trellis-quantized projections.

Every step runs a tree of nodes for each sequence through the model at once:
the projections (tf_rot_in_linear), the cache (tf_kv_write), the attention
(tf_tree_attention), the check of the drafts against the logits
(tf_verify_draft), and the cache rows of the accepted path (tf_kv_keep). A
tree of one node is ordinary decoding, and both give the same tokens.

The drafts come from a stand-in for a drafting model: the true continuation,
spoilt here and there, with a wrong sibling beside each.

    python examples/speculative_decode.py [--steps N]
"""

import argparse
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import trellis_quantized_linear_rot_gb300 as tf  # noqa: E402
from trellis_quantized_linear_rot_gb300 import synth  # noqa: E402

HIDDEN, HEADS, KV_HEADS, DIM, LAYERS, VOCAB, BITS, PAGE = 512, 8, 2, 64, 2, 1024, 4, 16
# Tree of a step: node 0 is the last token, 1-2-3-4 the drafted chain, and 5 to 8
# a sibling of each of those.
TREE = [-1, 0, 1, 2, 3, 0, 1, 2, 3]


class Projection:
    """One quantized projection with random weights, outputs of about unit size."""

    def __init__(self, n_in, n_out, seed):
        dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        self.n_out = n_out
        self.suh = dev(synth.make_scale(n_in, seed))
        self.svh = dev((synth.make_scale(n_out, seed + 1) * n_in ** -0.5).astype(np.float16))
        self.trellis = dev(synth.make_trellis(n_in, n_out, BITS, seed + 2).view(np.int32))

    def __call__(self, x, out_dtype=torch.float16):
        return tf.project(x, self.suh, self.trellis, self.svh, BITS, self.n_out, out_dtype=out_dtype)


class Model:
    def __init__(self, batch, capacity, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.embed = torch.randn((VOCAB, HIDDEN), device="cuda", generator=g).half()
        self.qkv = [Projection(HIDDEN, (HEADS + 2 * KV_HEADS) * DIM, 100 + 10 * i) for i in range(LAYERS)]
        self.out = [Projection(HEADS * DIM, HIDDEN, 200 + 10 * i) for i in range(LAYERS)]
        self.head = Projection(HIDDEN, VOCAB, 300)
        width = -(-capacity // PAGE)
        self.table = torch.randperm(batch * width, device="cuda", generator=g).to(torch.int32).view(batch, width)
        shape = (LAYERS, batch * width, PAGE, KV_HEADS, DIM)
        self.k, self.v = (torch.zeros(shape, dtype=torch.float16, device="cuda") for _ in range(2))

    def logits(self, tokens, parents, lengths):
        """Logits after every node of a tree of tokens [batch, nodes]."""
        b, n = tokens.shape
        x = self.embed[tokens.long()].view(b * n, HIDDEN)
        for i in range(LAYERS):
            rows = self.qkv[i](x).view(b, n, HEADS + 2 * KV_HEADS, DIM)
            q, k, v = rows.split([HEADS, KV_HEADS, KV_HEADS], dim=2)
            tf.tf_kv_write(k, v, self.k[i], self.v[i], self.table, lengths)
            o, _ = tf.tf_tree_attention(q, self.k[i], self.v[i], self.table, lengths, parents)
            x = x + self.out[i](o.view(b * n, HEADS * DIM))
            x = (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).half()
        return self.head(x, torch.float32).view(b, n, VOCAB)


def decode(model, first, count, parents, draft):
    """Decodes `count` tokens after `first` [batch]: (tokens [batch, count],
    steps). draft(done) gives the drafted tokens [batch, nodes - 1] when `done`
    [batch] tokens are out."""
    b = first.shape[0]
    tree = torch.tensor(parents, dtype=torch.int32, device="cuda")
    lengths = torch.zeros((b,), dtype=torch.int32, device="cuda")
    last = first.to(torch.int32)
    out = torch.zeros((b, count + len(parents)), dtype=torch.int32, device="cuda")
    done = torch.zeros((b,), dtype=torch.int64, device="cuda")
    steps = 0
    while int(done.min()) < count:
        # a sequence that has all its tokens sits out: an absent root, a negative length
        idle = done >= count
        tokens = torch.cat([last[:, None], draft(done)], dim=1).contiguous()
        here = torch.where(idle, torch.full_like(lengths, -1), lengths)
        trees = torch.where(idle[:, None], torch.full_like(tree, -2), tree).contiguous()
        logits = model.logits(tokens, trees, here)
        counts, path, new, _ = tf.tf_verify_draft(logits, tokens, trees, None, temperature=0.0)
        kept = tf.tf_kv_keep(model.k, model.v, model.table, here, path, counts)
        lengths = torch.where(idle, lengths, kept)
        at = done[:, None] + torch.arange(len(parents), device="cuda")
        fresh = torch.arange(len(parents), device="cuda") < counts[:, None]
        at = torch.where(fresh, at, torch.full_like(at, out.shape[1] - 1))
        out.scatter_(1, at, torch.where(fresh, new, torch.zeros_like(new)))
        end = (counts.long() - 1).clamp(min=0)
        last = torch.where(idle, last, new.gather(1, end[:, None])[:, 0])
        done = done + counts
        steps += 1
    tf.tf_device_error()
    return out[:, :count], steps


def stand_in_drafts(truth, seed):
    """Drafts for TREE from the known continuation: each chain token is right
    four times out of five, each sibling where the chain is wrong half the time."""
    rng = torch.Generator(device="cuda").manual_seed(seed)
    padded = torch.cat([truth, torch.zeros((truth.shape[0], 8), dtype=truth.dtype, device="cuda")], dim=1)

    def draft(done):
        ahead = padded.gather(1, done.clamp(max=truth.shape[1])[:, None] + torch.arange(4, device="cuda"))
        wrong = torch.randint(0, VOCAB, ahead.shape, device="cuda", generator=rng, dtype=torch.int32)
        u = torch.rand(ahead.shape, device="cuda", generator=rng)
        chain = torch.where(u < 0.8, ahead, wrong)
        sibling = torch.where(u > 0.9, ahead, (wrong + 1) % VOCAB)
        return torch.cat([chain, sibling], dim=1)

    return draft


def run(count=40, batch=3):
    first = torch.arange(1, batch + 1, device="cuda")
    capacity = count + 2 * len(TREE)
    none = lambda done: torch.zeros((batch, 0), dtype=torch.int32, device="cuda")  # noqa: E731
    plain, plain_steps = decode(Model(batch, capacity), first, count, [-1], none)
    spec, steps = decode(Model(batch, capacity), first, count, TREE, stand_in_drafts(plain, 7))
    return plain, plain_steps, spec, steps


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=40, help="tokens to decode for each sequence")
    plain, plain_steps, spec, steps = run(ap.parse_args().steps)
    print("one token a step: %d steps; a tree of %d nodes a step: %d steps" % (plain_steps, len(TREE), steps))
    print("the same tokens" if torch.equal(plain, spec) else "DIFFERENT TOKENS")
    print(spec[0].tolist())


if __name__ == "__main__":
    main()
