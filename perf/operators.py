"""Cases of the operators around the decode-row projections: the rows of a drafted token tree are written into
a paged cache, attend to it, are verified against the target's probabilities, and the accepted path is kept.

Where `own` is false, `run` computes each operator in its plain form, with elementary torch operations in 32
bits. Where it is true, it calls the package's entry points on the same state.

Conventions shared by all operators: a sequence's tree has `nodes` nodes; node 0 is the last accepted token
and the others are drafted ones; parents[j] < j is node j's parent, -1 marks a node without one, -2 an absent
node (padding). Node i's key and value sit in cache slot lengths[b] + i of the sequence, and slot s is row
s % page_size of page page_table[b][s // page_size].
"""

import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"fp16": 2, "bf16": 2, "fp32": 4}
HEAD_VOCAB = 129280   # outputs of the LM head this package serves


def listed():
    return [
        # One new token of one short conversation: the smallest call, where the launch counts. 40 heads of 128
        # are the LM head's 5,120 inputs.
        {"name": "attend 1 token", "op": "attend", "dtype": "fp16", "batch": 1, "nodes": 1, "kv_heads": 8, "group": 5,
         "dim": 128, "context": 300, "page": 16, "tree": "chain", "ragged": False},
        # A few conversations, each with a chain of four drafted tokens; a head layout without shared heads.
        {"name": "attend chains 16x64 heads", "op": "attend", "dtype": "bf16", "batch": 6, "nodes": 5, "kv_heads": 16,
         "group": 1, "dim": 64, "context": 1500, "page": 24, "tree": "chain", "ragged": True},
        # Ordinary serving without drafts: one token each of a full batch of long conversations.
        {"name": "attend batch of tokens", "op": "attend", "dtype": "bf16", "batch": 32, "nodes": 1, "kv_heads": 8,
         "group": 5, "dim": 128, "context": 8192, "page": 64, "tree": "chain", "ragged": True},
        # Speculative serving: a tree of 16 nodes for each sequence, some of them padded. 48 heads of 128 are the
        # 6,144 inputs of the wkv projection.
        {"name": "attend trees of 16", "op": "attend", "dtype": "fp16", "batch": 16, "nodes": 16, "kv_heads": 8,
         "group": 6, "dim": 128, "context": 4096, "page": 32, "tree": "tree", "ragged": True},
        # One long document with a wide tree: the case with the most arithmetic for each byte.
        {"name": "attend long tree of 64", "op": "attend", "dtype": "bf16", "batch": 1, "nodes": 64, "kv_heads": 8,
         "group": 5, "dim": 128, "context": 50001, "page": 128, "tree": "tree", "ragged": False},
        # Sampling one token of one sequence from its logits.
        {"name": "verify 1 row", "op": "verify", "dtype": "fp32", "batch": 1, "nodes": 1, "vocab": HEAD_VOCAB,
         "draft": False, "tree": "chain", "temperature": 0.8},
        # Chains of seven drafted tokens checked against the drafting model's own probabilities.
        {"name": "verify chains of 8", "op": "verify", "dtype": "bf16", "batch": 8, "nodes": 8, "vocab": HEAD_VOCAB,
         "draft": True, "tree": "chain", "temperature": 1.0},
        # A full batch of trees, a vocabulary that fills no whole vector.
        {"name": "verify trees of 16", "op": "verify", "dtype": "fp32", "batch": 32, "nodes": 16, "vocab": HEAD_VOCAB - 3,
         "draft": False, "tree": "tree", "temperature": 0.7},
        # The cache rows of one sequence's few new tokens, one layer.
        {"name": "write 5 tokens", "op": "write", "dtype": "fp16", "batch": 1, "nodes": 5, "kv_heads": 8, "group": 5,
         "dim": 128, "context": 2000, "page": 16},
        # The same for a full batch of wide trees.
        {"name": "write trees of 64", "op": "write", "dtype": "bf16", "batch": 64, "nodes": 64, "kv_heads": 8,
         "group": 6, "dim": 128, "context": 700, "page": 32},
        # The accepted path of one chain kept in one layer.
        {"name": "keep 1 path", "op": "keep", "dtype": "fp16", "batch": 1, "nodes": 8, "kv_heads": 8, "dim": 128,
         "context": 2000, "page": 16, "layers": 1},
        # The accepted paths of a full batch of trees, all layers of a model in one call.
        {"name": "keep paths of 32 layers", "op": "keep", "dtype": "bf16", "batch": 32, "nodes": 16, "kv_heads": 8,
         "dim": 128, "context": 500, "page": 64, "layers": 32},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 280.0)   # at rates of about 280 operations a byte


def draw(rng):
    while True:
        op = rng.choice(["attend", "attend", "verify", "verify", "write", "keep"])
        dtype = rng.choice(["fp16", "bf16"])
        kv_heads = rng.choice([1, 2, 4, 8, 16])
        group = rng.choice([1, 3, 4, 5, 6, 8])
        dim = rng.choice([64, 128])
        page = rng.choice([8, 16, 24, 32, 64, 128])
        tree = rng.choice(["chain", "tree"])
        nodes = _log_int(rng, 1, 64)
        if op == "attend":
            case = {"op": op, "dtype": dtype, "batch": _log_int(rng, 1, 32), "nodes": nodes, "kv_heads": kv_heads,
                    "group": group, "dim": dim, "context": _log_int(rng, 1, 50000), "page": page, "tree": tree,
                    "ragged": rng.random() < 0.7}
        elif op == "verify":
            case = {"op": op, "dtype": rng.choice(["fp16", "bf16", "fp32"]), "batch": _log_int(rng, 1, 32),
                    "nodes": _log_int(rng, 1, 24), "vocab": rng.choice([HEAD_VOCAB, rng.randint(2000, HEAD_VOCAB)]),
                    "draft": rng.random() < 0.5, "tree": tree,
                    "temperature": rng.choice([0.0, 0.6, 0.8, 1.0, 1.3])}
        elif op == "write":
            case = {"op": op, "dtype": dtype, "batch": _log_int(rng, 1, 64), "nodes": nodes, "kv_heads": kv_heads,
                    "group": group, "dim": dim, "context": _log_int(rng, 1, 2000), "page": page}
        else:
            case = {"op": op, "dtype": dtype, "batch": _log_int(rng, 1, 32), "nodes": _log_int(rng, 2, 32),
                    "kv_heads": kv_heads, "dim": dim, "context": _log_int(rng, 1, 1000), "page": page,
                    "layers": rng.choice([1, 1, 7, 32])}
        if _cost(case) <= max(_cost(c) for c in listed() if c["op"] == op):
            return case


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _rand(shape, g):
    return torch.rand(shape, device="cuda", generator=g)


def _lengths(case, g):
    """Context lengths: the case's own, or (ragged) from a quarter of it up to it."""
    b, c = case["batch"], case["context"]
    if not case.get("ragged", True):
        return torch.full((b,), c, dtype=torch.int32, device="cuda")
    lens = (c * (0.25 + 0.75 * _rand((b,), g))).to(torch.int32).clamp_(1, c)
    lens[0] = c
    return lens


def _parents(case, g):
    """A chain, or a tree whose node j hangs below one of the eight nodes before it; in a tree's batch every
    third sequence has its last nodes absent."""
    b, n = case["batch"], case["nodes"]
    j = torch.arange(n, device="cuda").expand(b, n)
    if case["tree"] == "chain":
        par = j - 1
    else:
        back = 1 + (_rand((b, n), g) * torch.clamp(j, max=8)).long()
        par = torch.clamp(j - back, min=0)
        par = torch.where(j == 0, torch.full_like(par, -1), par)
        absent = (torch.arange(b, device="cuda") % 3 == 2)[:, None] & (j >= max(1, n - n // 4))
        par = torch.where(absent, torch.full_like(par, -2), par)
    return par.to(torch.int32).contiguous()


def _cache(case, g, layers=None):
    """Page tables that scatter each sequence over the pool, and random caches."""
    b, page = case["batch"], case["page"]
    per = -(-(case["context"] + case["nodes"]) // page)
    pool = b * per + 3
    table = torch.randperm(pool, device="cuda", generator=g)[: b * per].to(torch.int32).view(b, per)
    shape = (pool, page, case["kv_heads"], case["dim"])
    if layers is not None:
        shape = (layers,) + shape
    dt = DTYPES[case["dtype"]]
    k = torch.randn(shape, device="cuda", dtype=dt, generator=g)
    v = torch.randn(shape, device="cuda", dtype=dt, generator=g)
    return table, k, v


def _logits(case, g):
    """Target logits with a broad background and a few plausible tokens a row, draft logits near them, and
    tokens drafted from the draft logits: drawn from them (draft) or its best ones in turn (no draft)."""
    b, n, v = case["batch"], case["nodes"], case["vocab"]
    target = torch.randn((b, n, v), device="cuda", generator=g)
    places = (_rand((b, n, 12), g) * v).long().clamp_(max=v - 1)
    target.scatter_add_(2, places, 6.0 + 8.0 * _rand((b, n, 12), g))
    draft = target + 0.5 * torch.randn((b, n, v), device="cuda", generator=g)
    par = _parents(case, g)
    up = par.long().clamp(min=0)
    t = max(case["temperature"], 0.3)
    if case["draft"]:   # one draw from the parent's draft probabilities: the largest of z + Gumbel noise
        rows = torch.gather(draft, 1, up[:, :, None].expand(b, n, v))
        rows = rows / t - torch.log(-torch.log(_rand((b, n, v), g).clamp_(1e-12, 1 - 1e-7)))
        tokens = rows.argmax(-1)
    else:               # the parent's best tokens, one for each of its children in turn
        k = min(n, v)
        best = torch.topk(draft, k, dim=-1).indices
        earlier = (up[:, None, :] == up[:, :, None]) & torch.ones((n, n), device="cuda", dtype=torch.bool).tril(-1)
        rank = (earlier & (torch.arange(n, device="cuda") > 0)).sum(-1).clamp_(max=k - 1)
        tokens = torch.gather(torch.gather(best, 1, up[:, :, None].expand(b, n, k)), 2, rank[:, :, None])[:, :, 0]
    return target, draft, par, tokens.to(torch.int32).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"case": case}
    b, n = case["batch"], case["nodes"]
    if op in ("attend", "write"):
        # q, k and v are parts of the rows that one fused projection gives.
        kh, d = case["kv_heads"], case["dim"]
        h = kh * case["group"]
        rows = torch.randn((b, n, (h + 2 * kh) * d), device="cuda", dtype=dt, generator=g)
        s["q"] = rows[:, :, : h * d].view(b, n, h, d)
        s["k_new"] = rows[:, :, h * d : (h + kh) * d].view(b, n, kh, d)
        s["v_new"] = rows[:, :, (h + kh) * d :].view(b, n, kh, d)
        s["lengths"] = _lengths(case, g)
        s["table"], s["k"], s["v"] = _cache(case, g)
    if op == "attend":
        s["parents"] = _parents(case, g)
        s["scale"] = 1.5 / math.sqrt(case["dim"])
    elif op == "verify":
        target, draft, s["parents"], s["tokens"] = _logits(case, g)
        s["logits"] = target.to(dt)
        s["draft"] = draft.to(dt) if case["draft"] else None
        s["u_accept"] = _rand((b, n), g) if case["draft"] else None
        s["u_sample"] = _rand((b, n), g)
        s["temperature"] = case["temperature"]
    elif op == "keep":
        s["lengths"] = _lengths(case, g)
        s["table"], s["k"], s["v"] = _cache(case, g, case["layers"])
        # A rising path from node 0, of a random length.
        steps = 1 + (_rand((b, n), g) * 2.5).long()
        path = torch.cumsum(steps, 1) - steps[:, :1]
        counts = torch.minimum(1 + (_rand((b,), g) * n).long(), (path < n).sum(1))
        keep = torch.arange(n, device="cuda")[None, :] < counts[:, None]
        s["path"] = torch.where(keep, path, torch.full_like(path, -1)).to(torch.int32)
        s["counts"] = counts.to(torch.int32)
    return s


# ------------------------------------------------------------- plain forms
def _slots(table, pos, page):
    """Row of the flattened pool (pages * page_size rows) for each position [batch, n]."""
    return torch.gather(table.long(), 1, pos // page) * page + pos % page


def _ancestors(parents):
    """[batch, node, node] truth values: column j is row i's own node or one of its ancestors."""
    b, n = parents.shape
    idx = torch.arange(n, device=parents.device)
    present = parents >= -1
    step = (parents[:, :, None] == idx) | (idx[:, None] == idx)
    step = (step & present[:, :, None]).float()
    reach = step
    for _ in range(max(1, math.ceil(math.log2(max(2, n))))):
        reach = (reach @ reach > 0).float()
    return (reach > 0) & present[:, :, None] & present[:, None, :]


def _plain_attend(s):
    case = s["case"]
    b, n, h, d = s["q"].shape
    kh, page = case["kv_heads"], case["page"]
    lens = s["lengths"].long()
    total = case["context"] + n                          # longest row of slots
    pos = torch.arange(total, device=lens.device).expand(b, total)
    where = _slots(s["table"], pos, page)
    k = s["k"].reshape(-1, kh, d)[where].float().permute(0, 2, 1, 3)   # [b, kh, total, d]
    v = s["v"].reshape(-1, kh, d)[where].float().permute(0, 2, 1, 3)
    q = s["q"].float().view(b, n, kh, h // kh, d).permute(0, 2, 1, 3, 4).reshape(b, kh, n * (h // kh), d)
    scores = (q @ k.transpose(2, 3)) * s["scale"]
    node = pos - lens[:, None]                           # tree node of a slot, negative in the context
    tree = torch.gather(_ancestors(s["parents"]), 2, node.clamp(0, n - 1)[:, None, :].expand(b, n, total))
    present = (s["parents"] >= -1)[:, :, None]
    seen = present & ((node < 0)[:, None, :] | ((node < n)[:, None, :] & tree))
    seen = seen[:, None, :, None, :].expand(b, kh, n, h // kh, total).reshape(b, kh, n * (h // kh), total)
    scores = torch.where(seen, scores, torch.full_like(scores, -math.inf))
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    e = torch.exp(scores - top)
    z = e.sum(-1, keepdim=True)
    o = (e @ v) / torch.where(z == 0, torch.ones_like(z), z)
    lse = (top + torch.log(z))[..., 0]
    o = o.view(b, kh, n, h // kh, d).permute(0, 2, 1, 3, 4).reshape(b, n, h, d)
    lse = lse.view(b, kh, n, h // kh).permute(0, 2, 1, 3).reshape(b, n, h)
    return o.to(s["q"].dtype), lse.contiguous()


def _weights(x, temperature):
    """z = x / T, e = exp(z - max z) and its whole-number weights w = round(2^30 e), with their exact sums."""
    z = x.float()
    z = torch.where(torch.isnan(z), torch.full_like(z, -math.inf), z)
    z = z * torch.tensor(1.0 / temperature if temperature > 0 else 1.0, dtype=torch.float32, device=x.device)
    top = z.amax(-1, keepdim=True)
    e = torch.where(z == top, (z > -math.inf).float(), torch.exp(z - top))
    w = torch.round(e * 2.0**30).to(torch.int64)
    return z, top, e, w, w.sum(-1)


def _pick(w, u):
    """The least index whose cumulative weight is above floor(u * total); -1 where there is no weight."""
    total = w.sum(-1)
    t = torch.minimum(torch.floor(u.double() * total.double()).long(), total - 1)
    return torch.where(total > 0, (torch.cumsum(w, -1) <= t[..., None]).sum(-1), torch.full_like(total, -1))


def _plain_verify(s):
    logits, tokens, par = s["logits"], s["tokens"].long(), s["parents"].long()
    b, n, v = logits.shape
    dev = logits.device
    rows = torch.arange(b, device=dev)
    z, top, e, w, mass = _weights(logits, s["temperature"])
    take = torch.full((b, n), -1, dtype=torch.int64, device=dev)   # the child a node goes on to
    inside = (tokens >= 0) & (tokens < v)
    if s["temperature"] > 0 and s["draft"] is not None:
        _, _, f, _, qmass = _weights(s["draft"], s["temperature"])
        unit = 2.0**61
        cp = (unit / mass.double()).float()
        level = torch.zeros((b, n), dtype=torch.float64, device=dev)                  # a
        left = torch.full((b, n), 2.0**31, dtype=torch.float64, device=dev)           # S
        spent = torch.zeros((b, n), dtype=torch.bool, device=dev)
        for c in range(1, n):
            x = par[:, c].clamp(min=0)
            t = tokens[:, c].clamp(0, v - 1)
            a, rest = level[rows, x], left[rows, x]
            pe, qe = e[rows, x], f[rows, x]
            cpx, q1 = cp[rows, x], unit / qmass[rows, x].double()
            pt, qt = pe[rows, t] * cpx, qe[rows, t] * q1.float()
            rt = torch.where(a > 0, (torch.round(pt) - torch.round(qe[rows, t] * (a * q1).float()).double()).clamp(min=0), pt.double())
            asked = (par[:, c] >= 0) & inside[:, c] & (take[rows, x] < 0) & ~spent[rows, x]
            ok = asked & (s["u_accept"][:, c].double() * qt.double() * rest < rt * 2.0**31)
            take[rows, x] = torch.where(ok, torch.full_like(x, c), take[rows, x])
            a1 = a + rest / 2.0**31
            res = torch.round(pe * cpx[:, None]).to(torch.int64) - torch.round(qe * (a1 * q1).float()[:, None]).to(torch.int64)
            s1 = res.clamp(min=0).sum(-1).double()
            no = asked & ~ok
            spent[rows, x] = spent[rows, x] | (no & (s1 == 0))
            level[rows, x] = torch.where(no, torch.where(s1 == 0, torch.zeros_like(a), a1), a)
            left[rows, x] = torch.where(no, s1, rest)
        node = torch.zeros((b,), dtype=torch.int64, device=dev)
        for _ in range(n):
            node = torch.where(take[rows, node] >= 0, take[rows, node], node)
        pe, qe, a = e[rows, node], f[rows, node], level[rows, node]
        q1 = unit / qmass[rows, node].double()
        res = torch.round(pe * cp[rows, node][:, None]).to(torch.int64) - torch.round(qe * (a * q1).float()[:, None]).to(torch.int64)
        end = _pick(torch.where(a[:, None] > 0, res.clamp(min=0), w[rows, node]), s["u_sample"][rows, node])
        pick = torch.full((b, n), -1, dtype=torch.int64, device=dev)
        pick[rows, node] = end
    else:
        pick = _pick(w, s["u_sample"]) if s["temperature"] > 0 else torch.where(mass > 0, z.argmax(-1), torch.full_like(mass, -1))
        for c in range(n - 1, 0, -1):     # the lowest matching child is written last
            x = par[:, c].clamp(min=0)
            ok = (par[:, c] >= 0) & inside[:, c] & (pick[rows, x] == tokens[:, c])
            take[rows, x] = torch.where(ok, torch.full_like(x, c), take[rows, x])
    counts = torch.zeros((b,), dtype=torch.int32, device=dev)
    path = torch.full((b, n), -1, dtype=torch.int32, device=dev)
    out = torch.full((b, n), -1, dtype=torch.int32, device=dev)
    logp = torch.zeros((b, n), dtype=torch.float32, device=dev)
    node = torch.zeros((b,), dtype=torch.int64, device=dev)
    going = par[:, 0] >= -1
    for k in range(n):
        nxt = take[rows, node]
        t = torch.where(nxt >= 0, tokens[rows, nxt.clamp(min=0)], pick[rows, node])
        lp = (z[rows, node, t.clamp(min=0)] - top[rows, node, 0]) - torch.log(mass[rows, node].float() * 2.0**-30)
        path[:, k] = torch.where(going, node.to(torch.int32), path[:, k])
        out[:, k] = torch.where(going, t.to(torch.int32), out[:, k])
        logp[:, k] = torch.where(going & (t >= 0), lp, logp[:, k])
        counts += going.to(torch.int32)
        going = going & (nxt >= 0)
        node = torch.where(nxt >= 0, nxt, node)
    return counts, path, out, logp


def _plain_write(s):
    b, n, kh, d = s["k_new"].shape
    pos = s["lengths"].long()[:, None] + torch.arange(n, device="cuda")
    where = _slots(s["table"], pos, s["case"]["page"])
    s["k"].view(-1, kh, d)[where] = s["k_new"]
    s["v"].view(-1, kh, d)[where] = s["v_new"]
    return s["k"], s["v"]


def _plain_keep(s):
    case = s["case"]
    n, kh, d = case["nodes"], case["kv_heads"], case["dim"]
    first = s["lengths"].long()[:, None]
    i = torch.arange(n, device="cuda")
    kept = i < s["counts"][:, None]
    to = _slots(s["table"], first + i, case["page"])
    come = _slots(s["table"], first + torch.where(kept, s["path"].long(), i), case["page"])
    for x in (s["k"], s["v"]):
        flat = x.view(case["layers"], -1, kh, d)
        flat[:, to] = flat[:, come]
    return s["k"], s["v"], s["lengths"] + s["counts"]


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"attend": _plain_attend, "verify": _plain_verify, "write": _plain_write, "keep": _plain_keep}[op](s)
    import trellis_quantized_linear_rot_gb300 as tf
    if op == "attend":
        return tf.tf_tree_attention(s["q"], s["k"], s["v"], s["table"], s["lengths"], s["parents"], scale=s["scale"])
    if op == "verify":
        return tf.tf_verify_draft(s["logits"], s["tokens"], s["parents"], s["u_sample"], temperature=s["temperature"],
                                  draft_logits=s["draft"], u_accept=s["u_accept"])
    if op == "write":
        tf.tf_kv_write(s["k_new"], s["v_new"], s["k"], s["v"], s["table"], s["lengths"])
        return s["k"], s["v"]
    return s["k"], s["v"], tf.tf_kv_keep(s["k"], s["v"], s["table"], s["lengths"], s["path"], s["counts"])


# -------------------------------------------------------------------- work
def work(case):
    op, e = case["op"], BYTES[case["dtype"]]
    b, n = case["batch"], case["nodes"]
    if op == "verify":
        rows = b * n * (2 if case["draft"] else 1)
        return {"bytes": rows * case["vocab"] * e + b * n * 32, "flops": rows * case["vocab"] * 4}
    slot = case["kv_heads"] * case["dim"] * e
    if op == "write":
        return {"bytes": 4 * b * n * slot, "flops": 0}
    if op == "keep":   # about a third of the nodes are kept, and their first stays where it is
        return {"bytes": 4 * case["layers"] * b * max(1, n // 3) * slot, "flops": 0}
    h = case["kv_heads"] * case["group"]
    slots = b * (case["context"] * (0.625 if case["ragged"] and b > 1 else 1.0) + n)
    return {"bytes": 2 * slots * slot + b * n * h * (2 * case["dim"] * e + 4) + slots / case["page"] * 4,
            "flops": 4 * n * h * case["dim"] * slots}


# ------------------------------------------------------------------- exact
def _exact_attend(case, s):
    b, n, h, d = s["q"].shape
    kh, group = case["kv_heads"], case["group"]
    page = case["page"]
    o = torch.zeros((b, n, h, d), dtype=torch.float64, device="cuda")
    lse = torch.full((b, n, h), -math.inf, dtype=torch.float64, device="cuda")
    lens, par = s["lengths"].tolist(), s["parents"].tolist()
    for i in range(b):
        count = lens[i] + n
        pages = s["table"][i, : -(-count // page)].long()
        k = s["k"][pages].reshape(-1, kh, d)[:count].double()
        v = s["v"][pages].reshape(-1, kh, d)[:count].double()
        hidden = torch.ones((n, n), dtype=torch.bool)
        for j in range(n):
            up = j if par[i][j] >= -1 else -1
            while up >= 0:
                hidden[j, up] = False
                up = par[i][up]
        hidden = hidden.cuda()
        for g in range(kh):
            q = s["q"][i, :, g * group : (g + 1) * group].double()
            sc = torch.einsum("nhd,sd->nhs", q, k[:, g]) * s["scale"]
            sc[:, :, lens[i] :] = sc[:, :, lens[i] :].masked_fill(hidden[:, None, :], -math.inf)
            live = [j for j in range(n) if par[i][j] >= -1]
            sc = sc[live]
            o[i, live, g * group : (g + 1) * group] = torch.einsum("nhs,sd->nhd", torch.softmax(sc, -1), v[:, g])
            lse[i, live, g * group : (g + 1) * group] = torch.logsumexp(sc, -1)
    return o, lse


def _exact_verify(case, s):
    b, n, v = s["logits"].shape
    t = case["temperature"]
    logp = torch.zeros((b, n), dtype=torch.float64, device="cuda")
    par, tok = s["parents"].tolist(), s["tokens"].tolist()
    for i in range(b):
        node, k = 0, 0
        while True:
            x = s["logits"][i, node].double() / (t if t > 0 else 1.0)
            p = torch.softmax(x, -1)
            children = [c for c in range(1, n) if par[i][c] == node]
            nxt = -1
            if t > 0 and case["draft"]:
                q = torch.softmax(s["draft"][i, node].double() / t, -1)
                r = p
                for c in children:
                    if float(s["u_accept"][i, c]) * float(q[tok[i][c]]) < float(r[tok[i][c]]):
                        nxt = c
                        break
                    r = (r - q).clamp(min=0)
                    r = r / r.sum()
                token = tok[i][nxt] if nxt >= 0 else int((torch.cumsum(r, 0) <= float(s["u_sample"][i, node])).sum().clamp(max=v - 1))
            else:
                token = int((torch.cumsum(p, 0) <= float(s["u_sample"][i, node])).sum().clamp(max=v - 1)) if t > 0 else int(x.argmax())
                match = [c for c in children if tok[i][c] == token]
                nxt = match[0] if match else -1
            logp[i, k] = torch.log_softmax(x, -1)[token]
            k += 1
            if nxt < 0:
                break
            node = nxt
    return None, None, None, logp


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _exact_attend(case, s)
    if case["op"] == "verify":
        return _exact_verify(case, s)
    return None   # copies: no computed numbers
