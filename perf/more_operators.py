"""Cases of the operators around a cache that is held in 4 or 8 bits: queries and keys are normed for each head and
rotated by their positions, keys and values are quantised as they are written into the paged cache, read back,
attended to, and the accepted path of a drafted tree is kept.

Where `own` is false, `run` computes each operator in its plain form, with elementary torch operations in 32
bits. Where it is true, it calls the package's entry points on the same state.

The cache: keys and values of one head and slot are head_dim whole numbers c of 4 or 8 bits (two in a byte, the
even element in the low half; stored with 8 or 128 added), and each row of them has a factor s in bf16: its values are
c * s. codes are [pages, page_size, kv_heads, head_dim * bits / 8] uint8, the factors of key and value [pages,
page_size, kv_heads, 2]. In memory the rows of one head and page lie together. Slot s of a sequence is row s %
page_size of page page_table[b][s // page_size]; a sequence's tree has `nodes` nodes in the slots after its
lengths[b] context tokens, and parents[j] < j is node j's parent (-1: none, -2: an absent node).
"""

import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
FAR = 131072          # positions go up to here


def listed():
    return [
        # One new token between the qkv projection and the cache: the smallest call, where the launch counts. 40 heads
        # of 128 are the LM head's 5,120 inputs.
        {"name": "norm 1 token", "op": "norm", "dtype": "fp16", "batch": 1, "nodes": 1, "kv_heads": 8, "group": 5,
         "dim": 128, "rotary": 128, "paired": False, "hadamard": False},
        # A prompt of 4,096 tokens before it is written in 4 bits: the rotation over the head spreads outliers. 48
        # heads of 128 are the 6,144 inputs of the wkv projection.
        {"name": "norm prompt", "op": "norm", "dtype": "bf16", "batch": 1, "nodes": 4096, "kv_heads": 8, "group": 6,
         "dim": 128, "rotary": 128, "paired": False, "hadamard": True},
        # The cache rows of one sequence's few new tokens, written and read back.
        {"name": "write 5 tokens", "op": "write", "dtype": "fp16", "bits": 4, "batch": 1, "nodes": 5, "kv_heads": 8,
         "group": 5, "dim": 128, "context": 2000, "page": 16},
        # Parts of 512 tokens of 16 prompts.
        {"name": "write parts of prompts", "op": "write", "dtype": "bf16", "bits": 8, "batch": 16, "nodes": 512,
         "kv_heads": 8, "group": 6, "dim": 128, "context": 3000, "page": 32},
        # One short conversation read back in 16 bits.
        {"name": "read 1 sequence", "op": "read", "dtype": "fp16", "bits": 8, "batch": 1, "kv_heads": 8, "dim": 128,
         "context": 300, "page": 16},
        # A batch of contexts of different lengths.
        {"name": "read batch", "op": "read", "dtype": "bf16", "bits": 4, "batch": 16, "kv_heads": 8, "dim": 128,
         "context": 4096, "page": 64},
        # One new token of one short conversation.
        {"name": "attend 1 token", "op": "attend", "dtype": "fp16", "bits": 4, "batch": 1, "nodes": 1, "kv_heads": 8,
         "group": 5, "dim": 128, "context": 300, "page": 16, "tree": "chain", "ragged": False},
        # A few conversations, each with a chain of four drafted tokens; a head layout without shared heads, 8 bits.
        {"name": "attend chains 16x64 heads", "op": "attend", "dtype": "bf16", "bits": 8, "batch": 6, "nodes": 5,
         "kv_heads": 16, "group": 1, "dim": 64, "context": 1500, "page": 24, "tree": "chain", "ragged": True},
        # Ordinary serving without drafts: one token each of a full batch of long conversations.
        {"name": "attend batch of tokens", "op": "attend", "dtype": "bf16", "bits": 4, "batch": 32, "nodes": 1,
         "kv_heads": 8, "group": 5, "dim": 128, "context": 8192, "page": 64, "tree": "chain", "ragged": True},
        # Speculative serving: a tree of 16 nodes for each sequence, some of them padded.
        {"name": "attend trees of 16", "op": "attend", "dtype": "fp16", "bits": 4, "batch": 16, "nodes": 16,
         "kv_heads": 8, "group": 6, "dim": 128, "context": 4096, "page": 32, "tree": "tree", "ragged": True},
        # The accepted path of one chain kept in one layer.
        {"name": "keep 1 path", "op": "keep", "dtype": "fp16", "bits": 4, "batch": 1, "nodes": 8, "kv_heads": 8,
         "dim": 128, "context": 2000, "page": 16, "layers": 1},
        # The accepted paths of a full batch of trees, all layers of a model in one call.
        {"name": "keep paths of 32 layers", "op": "keep", "dtype": "fp16", "bits": 8, "batch": 32, "nodes": 16,
         "kv_heads": 8, "dim": 128, "context": 500, "page": 64, "layers": 32},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 280.0)   # at rates of about 280 operations a byte


def draw(rng):
    while True:
        op = rng.choice(["norm", "write", "read", "attend", "attend", "attend", "keep"])
        case = {"op": op, "dtype": rng.choice(["fp16", "bf16"]), "kv_heads": rng.choice([1, 2, 3, 4, 8, 16]),
                "group": rng.choice([1, 3, 4, 5, 6, 8]), "dim": rng.choice([64, 128, 128, 256]),
                "page": rng.choice([8, 16, 24, 32, 64, 128]), "bits": rng.choice([4, 4, 8])}
        if op == "norm":
            case.update(batch=_log_int(rng, 1, 32), nodes=_log_int(rng, 1, 4096),
                        rotary=rng.choice([case["dim"], case["dim"], case["dim"] // 2, case["dim"] // 4]),
                        paired=rng.random() < 0.3, hadamard=rng.random() < 0.5)
        elif op == "write":
            case.update(batch=_log_int(rng, 1, 32), nodes=_log_int(rng, 1, 2048), context=_log_int(rng, 1, 3000))
        elif op == "read":
            case.update(batch=_log_int(rng, 1, 32), context=_log_int(rng, 1, 16384))
        elif op == "attend":
            case.update(batch=_log_int(rng, 1, 32), nodes=_log_int(rng, 1, 64), context=_log_int(rng, 1, 50000),
                        tree=rng.choice(["chain", "tree"]), ragged=rng.random() < 0.7)
        else:
            case.update(batch=_log_int(rng, 1, 32), nodes=_log_int(rng, 2, 32), context=_log_int(rng, 1, 1000),
                        layers=rng.choice([1, 1, 7, 32]))
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


def _rows(shape, dt, g):
    """Rows of a projection: heads of different sizes, a few dimensions much larger than the others."""
    x = torch.randn(shape, device="cuda", generator=g)
    h, d = shape[-2:]
    loud = 1.0 + 5.0 * (_rand((h, d), g) < 0.03).float()
    return (x * loud * (0.5 + _rand((h, 1), g))).to(dt)


def _cache(case, g, layers=None, extra=0):
    """Page tables that scatter each sequence over the pool, and caches of quantised rows."""
    b, page, kh, d, bits = case["batch"], case["page"], case["kv_heads"], case["dim"], case["bits"]
    per = -(-(case["context"] + case.get("nodes", 0) + extra) // page)
    pool = b * per + 3
    table = torch.randperm(pool, device="cuda", generator=g)[: b * per].to(torch.int32).view(b, per)
    lead = (pool,) if layers is None else (layers, pool)
    flat = math.prod(lead)
    codes, scales = [], []
    for _ in range(2):
        c = torch.empty((flat, kh, page, d * bits // 8), dtype=torch.uint8, device="cuda")
        s = torch.empty((flat, kh, page), dtype=torch.bfloat16, device="cuda")
        step = max(1, (1 << 26) // (kh * page * d))
        for i in range(0, flat, step):
            rows = _rows((page, min(step, flat - i), kh, d), torch.float32, g).permute(1, 2, 0, 3)
            whole, factor = _quantise(rows, bits)
            c[i : i + step], s[i : i + step] = _pack(whole, bits), factor[..., 0]
        codes.append(c.view(lead + c.shape[1:]).transpose(-3, -2))
        scales.append(s.view(lead + s.shape[1:]))
    return table, codes[0], codes[1], torch.stack(scales, -1).transpose(-3, -2)


def prepare(case, seed):
    g = _gen(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"case": case}
    b, n, kh, d = case["batch"], case.get("nodes", 0), case["kv_heads"], case["dim"]
    if op in ("norm", "write", "attend"):
        # q, k and v are parts of the rows that one fused projection gives.
        h = kh * case["group"]
        rows = _rows((b, n, h + 2 * kh, d), dt, g)
        s["q"], s["k_new"], s["v_new"] = rows[:, :, :h], rows[:, :, h : h + kh], rows[:, :, h + kh :]
    if op == "norm":
        r = case["rotary"]
        first = (_rand((b, 1), g) * (FAR - n)).to(torch.int32)
        s["positions"] = first + torch.arange(n, device="cuda", dtype=torch.int32)
        s["inv_freq"] = 500000.0 ** (-torch.arange(0, r, 2, dtype=torch.float64, device="cuda") / r)
        s["q_weight"], s["k_weight"] = (0.5 + _rand((2, d), g)).to(dt).unbind(0)
        s["q_out"] = torch.empty((b, n, h, d), dtype=dt, device="cuda")
        s["k_out"] = torch.empty((b, n, kh, d), dtype=dt, device="cuda")
        return s
    s["lengths"] = _lengths(case, g)
    s["table"], s["k"], s["v"], s["scales"] = _cache(case, g, case.get("layers"))
    if op == "write":
        s["new_lengths"] = s["lengths"] + n
        s["k_out"], s["v_out"] = (torch.zeros((b, n, kh, d), dtype=dt, device="cuda") for _ in range(2))
    elif op == "read":
        s["k_out"], s["v_out"] = (torch.zeros((b, case["context"], kh, d), dtype=dt, device="cuda") for _ in range(2))
    elif op == "attend":
        s["parents"] = _parents(case, g)
        s["scale"] = 1.0 / math.sqrt(d)
        s["out"] = torch.empty((b, n, h, d), dtype=dt, device="cuda")
        s["lse"] = torch.empty((b, n, h), dtype=torch.float32, device="cuda")
    else:
        # A rising path from node 0, of a random length.
        steps = 1 + (_rand((b, n), g) * 2.5).long()
        path = torch.cumsum(steps, 1) - steps[:, :1]
        counts = torch.minimum(1 + (_rand((b,), g) * n).long(), (path < n).sum(1))
        keep = torch.arange(n, device="cuda")[None, :] < counts[:, None]
        s["path"] = torch.where(keep, path, torch.full_like(path, -1)).to(torch.int32)
        s["counts"] = counts.to(torch.int32)
        s["kept_lengths"] = torch.empty_like(s["lengths"])
    return s


# ------------------------------------------------------------- plain forms
def _quantise(x, bits):
    """Whole numbers and factors of rows x [..., head_dim]."""
    most = 7.0 if bits == 4 else 127.0
    s = (x.abs().amax(-1, keepdim=True) / most).to(torch.bfloat16)
    f = s.float()
    whole = torch.round(x / torch.where(f == 0, torch.ones_like(f), f)).clamp(-most, most)
    return torch.where(f == 0, torch.zeros_like(whole), whole), s


def _pack(whole, bits):
    if bits == 8:
        return (whole + 128.0).to(torch.uint8)
    u = (whole + 8.0).to(torch.uint8)
    return u[..., 0::2] | (u[..., 1::2] << 4)


def _values(codes, s, bits):
    """fp32 values of packed rows."""
    if bits == 8:
        whole = codes.float() - 128.0
    else:
        whole = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float() - 8.0
    return whole * s.float()[..., None]


def _slots(table, pos, page):
    """Row of the flattened pool (pages * page_size rows) for each position [batch, n]."""
    return table.long().gather(1, pos // page), pos % page


def _ancestors(parents):
    """[batch, node, node] truth values: column j is row i's own node or one of its ancestors."""
    b, n = parents.shape
    idx = torch.arange(n, device=parents.device)
    present = parents >= -1
    step = (parents[:, :, None] == idx) | (idx[:, None] == idx)
    reach = (step & present[:, :, None]).float()
    for _ in range(max(1, math.ceil(math.log2(max(2, n))))):
        reach = (reach @ reach > 0).float()
    return (reach > 0) & present[:, :, None] & present[:, None, :]


def _signs(d):
    """The Sylvester-Hadamard matrix: (-1) to the number of ones that i and j share."""
    i = torch.arange(d, device="cuda")
    both = i[:, None] & i
    ones = (both[..., None] >> torch.arange(9, device="cuda") & 1).sum(-1)
    return 1.0 - 2.0 * (ones % 2).float()


def _normed(x, weight, s):
    case = s["case"]
    r, d = case["rotary"], case["dim"]
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    angle = s["positions"].double()[:, :, None, None] * s["inv_freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if case["paired"]:
        a, c = y[..., 0:r:2], y[..., 1:r:2]
        turned = torch.stack([a * cos - c * sin, c * cos + a * sin], -1).flatten(-2)
    else:
        a, c = y[..., : r // 2], y[..., r // 2 : r]
        turned = torch.cat([a * cos - c * sin, c * cos + a * sin], -1)
    y = torch.cat([turned, y[..., r:]], -1)
    if case["hadamard"]:
        y = (y @ _signs(d)) * (1.0 / math.sqrt(d))
    return y.to(x.dtype)


def _plain_norm(s):
    return _normed(s["q"], s["q_weight"], s), _normed(s["k_new"], s["k_weight"], s)


def _plain_write(s):
    case = s["case"]
    b, n = s["k_new"].shape[:2]
    pos = s["lengths"].long()[:, None] + torch.arange(n, device="cuda")
    pg, row = _slots(s["table"], pos, case["page"])
    ks, vs = _quantise(s["k_new"].float(), case["bits"]), _quantise(s["v_new"].float(), case["bits"])
    s["k"][pg, row], s["v"][pg, row] = _pack(ks[0], case["bits"]), _pack(vs[0], case["bits"])
    s["scales"][pg, row] = torch.cat([ks[1], vs[1]], -1)
    factors = s["scales"][pg, row]
    return tuple(_values(c[pg, row], factors[..., i], case["bits"]).to(s["k_new"].dtype)
                 for i, c in enumerate((s["k"], s["v"])))


def _plain_read(s):
    case = s["case"]
    b, c = case["batch"], case["context"]
    pos = torch.arange(c, device="cuda").expand(b, c)
    pg, row = _slots(s["table"], pos, case["page"])
    there = (pos < s["lengths"][:, None])[..., None, None]
    factors = s["scales"][pg, row]
    return tuple(torch.where(there, _values(x[pg, row], factors[..., i], case["bits"]).to(o.dtype), o)
                 for i, (x, o) in enumerate(((s["k"], s["k_out"]), (s["v"], s["v_out"]))))


def _plain_attend(s):
    case = s["case"]
    b, n, h, d = s["q"].shape
    kh, page = case["kv_heads"], case["page"]
    lens = s["lengths"].long()
    total = case["context"] + n                          # longest row of slots
    pos = torch.arange(total, device=lens.device).expand(b, total)
    pg, row = _slots(s["table"], pos, page)
    factors = s["scales"][pg, row]
    k = _values(s["k"][pg, row], factors[..., 0], case["bits"]).permute(0, 2, 1, 3)   # [b, kh, total, d]
    v = _values(s["v"][pg, row], factors[..., 1], case["bits"]).permute(0, 2, 1, 3)
    q = s["q"].float().reshape(b, n, kh, h // kh, d).permute(0, 2, 1, 3, 4).reshape(b, kh, n * (h // kh), d)
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


def _plain_keep(s):
    case = s["case"]
    first = s["lengths"].long()[:, None]
    i = torch.arange(case["nodes"], device="cuda")
    kept = i < s["counts"][:, None]
    to = _slots(s["table"], first + i, case["page"])
    come = _slots(s["table"], first + torch.where(kept, s["path"].long(), i), case["page"])
    for x in (s["k"], s["v"], s["scales"]):
        x[:, to[0], to[1]] = x[:, come[0], come[1]]
    return s["k"], s["v"], s["scales"], s["lengths"] + s["counts"]


def run(s):
    op = s["case"]["op"]
    if not own:
        return {"norm": _plain_norm, "write": _plain_write, "read": _plain_read, "attend": _plain_attend,
                "keep": _plain_keep}[op](s)
    import trellis_quantized_linear_rot_gb300 as tf
    if op == "norm":
        return tf.tf_qk_norm_rope(s["q"], s["k_new"], s["positions"], s["inv_freq"], s["q_weight"], s["k_weight"],
                                  eps=1e-6, interleaved=s["case"]["paired"], hadamard=s["case"]["hadamard"],
                                  q_out=s["q_out"], k_out=s["k_out"])
    if op == "write":   # what is held in 4 or 8 bits is read back as the values it stands for
        tf.tf_kvq_write(s["k_new"], s["v_new"], s["k"], s["v"], s["scales"], s["table"], s["lengths"])
        return tf.tf_kvq_read(s["k"], s["v"], s["scales"], s["table"], s["new_lengths"], starts=s["lengths"],
                              k_out=s["k_out"], v_out=s["v_out"])
    if op == "read":
        return tf.tf_kvq_read(s["k"], s["v"], s["scales"], s["table"], s["lengths"], k_out=s["k_out"],
                              v_out=s["v_out"])
    if op == "attend":
        return tf.tf_kvq_attention(s["q"], s["k"], s["v"], s["scales"], s["table"], s["lengths"], s["parents"],
                                   scale=s["scale"], out=s["out"], lse=s["lse"])
    # (a move of rows: the bytes themselves have to be the same)
    return s["k"], s["v"], s["scales"], tf.tf_kvq_keep(s["k"], s["v"], s["scales"], s["table"], s["lengths"],
                                                       s["path"], s["counts"], new_lengths=s["kept_lengths"])


# -------------------------------------------------------------------- work
def work(case):
    op, b, n, kh, d = case["op"], case["batch"], case.get("nodes", 0), case["kv_heads"], case["dim"]
    if op == "norm":
        elements = b * n * kh * (case["group"] + 1) * d
        return {"bytes": 4 * elements + 4 * b * n, "flops": elements * (8 + (math.log2(d) if case["hadamard"] else 0))}
    row = 2 * d * case["bits"] // 8 + 4      # key, value and their factors, of one head and slot
    if op == "write":                        # 16-bit rows in, cache rows out, and back
        return {"bytes": b * n * kh * (4 * d + row + row + 4 * d), "flops": 12 * b * n * kh * d}
    mean = 0.625 if case.get("ragged", True) and b > 1 else 1.0
    if op == "read":
        slots = b * case["context"] * mean
        return {"bytes": slots * kh * (row + 4 * d), "flops": 4 * slots * kh * d}
    if op == "keep":   # about a third of the nodes are kept, and their first stays where it is
        return {"bytes": 2 * case["layers"] * b * max(1, n // 3) * kh * row, "flops": 0}
    h = kh * case["group"]
    slots = b * (case["context"] * mean + n)
    return {"bytes": slots * kh * row + b * n * h * (4 * d + 4) + slots / case["page"] * 4,
            "flops": 4 * n * h * d * slots}


# ------------------------------------------------------------------- exact
def _held(codes, factor, bits):
    """64-bit values of rows as they are held."""
    x = codes.to(torch.int64)
    if bits == 4:
        x = torch.cat([(x % 16)[..., None], (x // 16)[..., None]], -1).reshape(x.shape[:-1] + (-1,))
    return (x - 2 ** (bits - 1)).double() * factor.double()[..., None]


def _exact_norm(case, s):
    out = []
    d, r = case["dim"], case["rotary"]
    signs = torch.ones((1, 1), dtype=torch.float64, device="cuda")
    while signs.shape[0] < d:
        signs = torch.cat([torch.cat([signs, signs], 1), torch.cat([signs, -signs], 1)], 0)
    for x, w in ((s["q"], s["q_weight"]), (s["k_new"], s["k_weight"])):
        y = x.double()
        y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / d + 1e-6) * w.double()
        first = torch.arange(0, r, 2, device="cuda") if case["paired"] else torch.arange(r // 2, device="cuda")
        second = first + (1 if case["paired"] else r // 2)
        turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"),
                           s["positions"].double()[..., None, None] * s["inv_freq"])
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        out.append(y @ signs / math.sqrt(d) if case["hadamard"] else y)
    return tuple(out)


def _exact_write(case, s):
    """Row by row: the factor is the definition's, a whole number is the nearest one to x / s."""
    most = 2 ** (case["bits"] - 1) - 1
    out = []
    for x in (s["k_new"], s["v_new"]):
        x = x.double()
        f = (x.abs().max(-1, keepdim=True).values.float() / most).bfloat16().double()
        out.append(torch.round(x / torch.where(f > 0, f, 1.0)).clamp(-most, most) * f)
    return tuple(out)


def _exact_read(case, s):
    out = []
    for i, (x, o) in enumerate(((s["k"], s["k_out"]), (s["v"], s["v_out"]))):
        o = o.double()
        for j, count in enumerate(s["lengths"].tolist()):
            pages = s["table"][j, : -(-count // case["page"])].long()
            rows = _held(x[pages], s["scales"][pages][..., i], case["bits"])
            o[j, :count] = rows.reshape(-1, case["kv_heads"], case["dim"])[:count]
        out.append(o)
    return tuple(out)


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
        k, v = (_held(x[pages], s["scales"][pages][..., j], case["bits"]).reshape(-1, kh, d)[:count]
                for j, x in enumerate((s["k"], s["v"])))
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


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "keep":
        return None   # copies: no computed numbers
    return {"norm": _exact_norm, "write": _exact_write, "read": _exact_read, "attend": _exact_attend}[case["op"]](case, s)
