"""Greedy decoding with a tree of drafted tokens, on a small synthetic model of
trellis-quantized projections.

Every step runs a tree of nodes for each sequence through the model at once:
the projections (tf_rot_in_linear), the cache (tf_kv_write), the attention
(tf_tree_attention), the check of the drafts against the logits
(tf_verify_draft), and the cache rows of the accepted path (tf_kv_keep). A
tree of one node is ordinary decoding, and with a cache of 16 bits both give
the same tokens.

The drafts come from a stand-in for a drafting model: the true continuation,
spoilt here and there, with a wrong sibling beside each.

With --cache 4 or 8 queries and keys are normed and rotated by their positions
(tf_qk_norm_rope), and the cache is held in that many bits (tf_kvq_write,
tf_kvq_attention, tf_kvq_keep). Two ways of summing that differ in the last bit
may round a cache row differently then, so that tokens can come apart where
two logits are close.

    python examples/speculative_decode.py [--steps N] [--cache 4]
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
    def __init__(self, batch, capacity, seed=0, cache_bits=None):
        self.cache_bits = cache_bits
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.embed = torch.randn((VOCAB, HIDDEN), device="cuda", generator=g).half()
        self.qkv = [Projection(HIDDEN, (HEADS + 2 * KV_HEADS) * DIM, 100 + 10 * i) for i in range(LAYERS)]
        self.out = [Projection(HEADS * DIM, HIDDEN, 200 + 10 * i) for i in range(LAYERS)]
        self.head = Projection(HIDDEN, VOCAB, 300)
        width = -(-capacity // PAGE)
        self.table = torch.randperm(batch * width, device="cuda", generator=g).to(torch.int32).view(batch, width)
        if cache_bits:
            self.k, self.v, self.scales = tf.tf_kvq_cache(batch * width, PAGE, KV_HEADS, DIM, cache_bits, layers=LAYERS)
            self.inv_freq = 10000.0 ** (-torch.arange(0, DIM, 2, dtype=torch.float64, device="cuda") / DIM)
        else:
            shape = (LAYERS, batch * width, PAGE, KV_HEADS, DIM)
            self.k, self.v = (torch.zeros(shape, dtype=torch.float16, device="cuda") for _ in range(2))

    def logits(self, tokens, parents, lengths):
        """Logits after every node of a tree of tokens [batch, nodes]."""
        b, n = tokens.shape
        x = self.embed[tokens.long()].view(b * n, HIDDEN)
        for i in range(LAYERS):
            rows = self.qkv[i](x).view(b, n, HEADS + 2 * KV_HEADS, DIM)
            q, k, v = rows.split([HEADS, KV_HEADS, KV_HEADS], dim=2)
            o = self.attend(i, q, k, v, parents, lengths)
            x = x + self.out[i](o.view(b * n, HEADS * DIM))
            x = (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).half()
        return self.head(x, torch.float32).view(b, n, VOCAB)

    def attend(self, i, q, k, v, parents, lengths):
        """The tree's keys and values into layer i's cache, and its attention."""
        if not self.cache_bits:
            tf.tf_kv_write(k, v, self.k[i], self.v[i], self.table, lengths)
            return tf.tf_tree_attention(q, self.k[i], self.v[i], self.table, lengths, parents)[0]
        depth = torch.tensor(depths(q.shape[1]), dtype=torch.int32, device="cuda")
        # (an idle sequence's length is negative, and with it its positions: nothing of it is written)
        positions = torch.where(lengths[:, None] < 0, lengths[:, None], lengths[:, None] + depth)
        q, k = tf.tf_qk_norm_rope(q, k, positions, self.inv_freq, hadamard=True)
        cache = (self.k[i], self.v[i], self.scales[i], self.table, lengths)
        tf.tf_kvq_write(k, v, *cache)
        return tf.tf_kvq_attention(q, *cache, parents)[0]

    def keep(self, lengths, path, counts):
        """The accepted path kept in all layers; the new lengths."""
        if not self.cache_bits:
            return tf.tf_kv_keep(self.k, self.v, self.table, lengths, path, counts)
        return tf.tf_kvq_keep(self.k, self.v, self.scales, self.table, lengths, path, counts)


def depths(nodes):
    """Steps from node 0 to each node of TREE, or of a tree of one node."""
    out = []
    for j in range(nodes):
        out.append(0 if TREE[j] < 0 else out[TREE[j]] + 1)
    return out


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
        kept = model.keep(here, path, counts)
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


def run(count=40, batch=3, cache_bits=None):
    first = torch.arange(1, batch + 1, device="cuda")
    capacity = count + 2 * len(TREE)
    none = lambda done: torch.zeros((batch, 0), dtype=torch.int32, device="cuda")  # noqa: E731
    plain, plain_steps = decode(Model(batch, capacity, cache_bits=cache_bits), first, count, [-1], none)
    spec, steps = decode(Model(batch, capacity, cache_bits=cache_bits), first, count, TREE, stand_in_drafts(plain, 7))
    return plain, plain_steps, spec, steps


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--steps", type=int, default=40, help="tokens to decode for each sequence")
    ap.add_argument("--cache", type=int, choices=(4, 8), help="bits of the cache (16 without this)")
    args = ap.parse_args()
    plain, plain_steps, spec, steps = run(args.steps, cache_bits=args.cache)
    print("one token a step: %d steps; a tree of %d nodes a step: %d steps" % (plain_steps, len(TREE), steps))
    if args.cache:
        print("%d of %d tokens alike" % (int((plain == spec).sum()), plain.numel()))
    else:
        print("the same tokens" if torch.equal(plain, spec) else "DIFFERENT TOKENS")
    print(spec[0].tolist())


if __name__ == "__main__":
    main()
