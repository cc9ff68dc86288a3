"""Plain 64-bit forms of the operators of tf_spec.h, and what may separate a
kernel's outputs from them. Written from the definitions, on the CPU in numpy;
they share no code with the kernels or the binding."""

import numpy as np

UNIT = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}   # bound of one rounding's relative error


def slot_rows(table_row, page_size, count):
    s = np.arange(count)
    return np.asarray(table_row)[s // page_size].astype(np.int64), s % page_size


def seen_nodes(parents):
    """[n, n] truth values: row i sees node j. Absent nodes see and are seen by none."""
    n = len(parents)
    out = np.zeros((n, n), dtype=bool)
    for i in range(n):
        j = i
        while 0 <= j < n and parents[j] >= -1 and (j == i or parents[j] < n):
            out[i, j] = True
            j = parents[j]
    return out


def attend(q, k, v, seen, scale):
    """One sequence: q [n, h, d], k and v [slots, kh, d], seen [n, slots].
    Returns out, lse, and per element the mean magnitude sum p |v| that the
    weights' rounding scales with, and per row the bound of a score's error."""
    n, h, d = q.shape
    group = h // k.shape[1]
    out, mag = np.zeros((n, h, d)), np.zeros((n, h, d))
    lse, err = np.full((n, h), -np.inf), np.zeros((n, h))
    for i in range(n):
        cols = np.flatnonzero(seen[i])
        if not len(cols):
            continue
        for x in range(h):
            kk, vv = k[cols, x // group], v[cols, x // group]
            s = scale * (kk @ q[i, x])
            top = s.max()
            if top == -np.inf:
                continue
            p = np.exp(s - top)
            z = p.sum()
            out[i, x] = p @ vv / z
            mag[i, x] = p @ np.abs(vv) / z
            lse[i, x] = top + np.log(z)
            # fp32: d products summed in any order, one product with the scale
            err[i, x] = (d + 2) * 2.0 ** -24 * np.abs(scale) * (np.abs(kk) @ np.abs(q[i, x])).max()
    return out, lse, mag, err


def attend_bounds(out, lse, mag, err, dtype, slots):
    """Largest |difference| allowed: a score error e moves every weight by a
    factor exp(+-e) (twice: weight and sum), the weights are rounded to the
    dtype (relative unit u, or 2^-25 absolute in fp16's subnormals) and so is
    the result; the fp32 sums add slots * 2^-24 at most, exp 2^-22."""
    u = UNIT[dtype]
    rel = 2 * err[..., None] + u + slots * 2.0 ** -24 + 2.0 ** -21
    tiny = slots * 2.0 ** -25 * 8 + 2.0 ** -24 if dtype == "fp16" else 0.0
    # exp(2e) - 1 <= 2.2 e for e up to 0.08
    return 1.1 * rel * mag + u * np.abs(out) + tiny + 1e-30, \
        1.1 * err + slots * 2.0 ** -24 + 2.0 ** -21 * (1 + np.abs(np.where(np.isfinite(lse), lse, 0)))


def soft(x):
    """Probabilities of a row as the definition has them (NaN counts as -inf)."""
    x = np.where(np.isnan(x), -np.inf, np.asarray(x, dtype=np.float64))
    top = x.max()
    if top == -np.inf:
        return None
    e = np.where(x == top, 1.0, 0.0) if top == np.inf else np.exp(x - top)
    return e / e.sum()


def may_pick(p, u, delta):
    """Tokens the cumulative rule may give when sums are off by up to delta."""
    u = min(max(u if u == u else 0.0, 0.0), 1.0)
    cum = np.cumsum(p)
    low = np.concatenate([[0.0], cum[:-1]])
    last = np.flatnonzero(p > 0)[-1]
    return (cum > u - delta) & ((low <= u + delta) | (np.arange(len(p)) == last)) & \
        ((np.arange(len(p)) <= last)) & (p > -1)


def check_walk(logits, tokens, parents, u_sample, temperature, draft, u_accept, got, seq=""):
    """Follows a kernel's answer for one sequence down the tree and asserts
    that every decision is one the definition allows, with probabilities off
    by at most delta. got = (count, path, out_tokens, logprobs)."""
    n, vocab = logits.shape
    count, path, out, logp = got
    t = temperature if temperature > 0 else 1.0
    ok_par = [p if p < j else -2 for j, p in enumerate(parents)]
    if ok_par[0] < -1:
        assert count == 0 and np.all(path == -1) and np.all(out == -1) and np.all(logp == 0), seq
        return
    assert 1 <= count <= n, seq
    assert np.all(path[count:] == -1) and np.all(out[count:] == -1) and np.all(logp[count:] == 0), seq
    node = 0
    for k in range(count):
        where = "%s step %d node %d" % (seq, k, node)
        assert path[k] == node, where
        x = np.where(np.isnan(logits[node]), -np.inf, logits[node].astype(np.float64)) / t
        p = soft(x)
        kids = [c for c in range(node + 1, n) if ok_par[c] == node and 0 <= tokens[c] < vocab]
        last = k == count - 1
        token = out[k]
        if p is None:
            assert last and token == -1 and logp[k] == 0, where
            return
        top = x[np.isfinite(x)].max() if np.isfinite(x).any() else 0.0
        low = np.abs(x[np.isfinite(x)]).max() if np.isfinite(x).any() else 0.0
        # fp32 rounding of z and of z - max, exp's two places, the whole-number grid
        delta = (3 * low + abs(top) + 4) * 2.0 ** -23 + vocab * 2.0 ** -31
        assert 0 <= token < vocab, where
        want = np.log(p[token]) if p[token] > 0 else None
        if want is not None and np.isfinite(x[token]):
            assert abs(logp[k] - want) <= 4 * delta + 2.0 ** -22 * abs(want), (where, logp[k], want)
        if not last:
            nxt = path[k + 1]
            assert nxt in kids and tokens[nxt] == token, where
        if temperature == 0:
            assert token == int(np.argmax(x)), where
            match = [c for c in kids if tokens[c] == token]
            assert (not match) if last else (match and match[0] == nxt), where
        elif draft is None:
            assert may_pick(p, u_sample[node], delta)[token], (where, token)
            match = [c for c in kids if tokens[c] == token]
            assert (not match) if last else (match and match[0] == nxt), where
        else:
            q = soft(draft[node].astype(np.float64) / t)
            q = np.zeros(vocab) if q is None else q
            zd = draft[node].astype(np.float64) / t
            zd = np.abs(zd[np.isfinite(zd)]).max() if np.isfinite(zd).any() else 0.0
            dd = delta + (4 * zd + 4) * 2.0 ** -23 + vocab * 2.0 ** -31
            r, slack, whole = p, dd, True
            for c in kids:
                tk = tokens[c]
                lhs, rhs = u_accept[c] * q[tk], r[tk]
                if not last and c == nxt:
                    assert lhs < rhs + slack, (where, c)
                    break
                assert lhs >= rhs - slack, (where, c)
                rest = np.maximum(r - q, 0)
                mass = rest.sum()
                if mass <= 4 * slack:
                    return   # too little is left to tell: tested on its own
                r, slack, whole = rest / mass, 3 * slack / mass, False
            else:
                assert last, where
                assert may_pick(r, u_sample[node], slack * (1 if whole else 2))[token], (where, token)
        node = path[k + 1] if not last else node
