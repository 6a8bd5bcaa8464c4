"""Plain definitions of the rotation, of the edits of logits and of the acceptance of trees, in 64 bits, with the errors
that fp32 arithmetic and one rounding to the type allow."""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # half a step, relative
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}   # half a step of the smallest


def frequencies(R, base=10000.0, scaling=None):
    s = scaling or {}
    kind, out = s.get("kind"), []
    if kind == "ntk" and R > 2:
        base = base * s["factor"] ** (R / (R - 2))
    for i in range(R // 2):
        f = base ** (-2 * i / R)
        if kind == "linear":
            f /= s["factor"]
        if kind == "parts":
            g = min(1, max(0, (s["original"] * f / (2 * math.pi) - s["low"]) / (s["high"] - s["low"])))
            f = g * f + (1 - g) * f / s["factor"]
        out.append(f)
    return out


def rotate_reference(x, positions, freq, inter=False, gain=1.0, norm=False, w=None, eps=1e-6):
    """x [N, H, D] (any type), positions [N]: the result in 64 bits, and the error it may have before the rounding to the
    type.  Angles are reduced with Python's integers: a frequency is a fraction, positions are whole numbers."""
    from fractions import Fraction
    x = x.double()
    N, H, D = x.shape
    R = 2 * len(freq)
    rel = 0.0
    if norm:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps)
        if w is not None:
            x = x * w.double()
        # D squares summed in fp32 (a step each, halved by the root), root, products: 2^-24 each
        rel = (D / 2 + 8) * 2.0 ** -24
    y, err = x.clone(), rel * x.abs()
    if R:
        two_pi = Fraction(math.pi) * 2 + Fraction(1.2246467991473532e-16) * 2      # pi to 106 bits
        turns = [Fraction(f) / two_pi for f in freq]
        angle = torch.tensor([[float((p * t) % 1) for t in turns] for p in positions.tolist()], dtype=torch.float64) * 2 * math.pi
        angle = angle.to(x.device)
        c, s = torch.cos(angle)[:, None] * gain, torch.sin(angle)[:, None] * gain
        ia = torch.arange(0, R, 2) if inter else torch.arange(0, R // 2)
        ib = ia + (1 if inter else R // 2)
        a, b = x[..., ia], x[..., ib]
        y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
        # sine and cosine: half turns in fp32 (pi 2^-24) and the functions themselves (2^-22); two products, a sum
        e = abs(gain) * (a.abs() + b.abs()) * (rel + 2.0 ** -21 + 4 * 2.0 ** -24)
        err[..., ia], err[..., ib] = e, e
    return y, err


def assert_rounded(got, y, err, what=""):
    """got: the type's values of y, rounded once, within err."""
    tol = 1.01 * U[got.dtype] * (y.abs() + err) + err + TINY[got.dtype]
    off = (got.double().to(y.device) - y).abs()
    assert (off <= tol).all(), (what, float((off / tol).max()), float(off.max()))


def depth(mask_row, b):
    return bin(mask_row & ((1 << b) - 1)).count("1")


def to_mask(rows):
    """Rows of Python integers as the int64 tensor that the calls take."""
    return torch.tensor([[m - (1 << 64) if m >> 63 else m for m in row] for row in rows], dtype=torch.int64)


def random_trees(S, B, rng):
    masks = []
    for _ in range(S):
        seen = [1]
        for b in range(1, B):
            seen.append(seen[rng.randrange(b)] | (1 << b))
        masks.append(seen)
    return masks


def edit_reference(logits, tokens=None, masks=None, lengths=None, history=None, prompt=None, repetition=None, frequency=None,
                   presence=None, bias=None, allowed=None):
    """logits [S, B, V] on the CPU; history, prompt: lists of tokens (prompt: how many of them); bias: per stream a list of
    (token, value); allowed: [S][B] sets or None.  Returns the edited logits in 64 bits and the error that fp32 allows."""
    S, B, V = logits.shape
    z = logits.double().clone()
    err = torch.zeros_like(z)
    for s in range(S):
        r, f, p = (1.0 if repetition is None else float(repetition[s]), 0.0 if frequency is None else float(frequency[s]),
                   0.0 if presence is None else float(presence[s]))
        for b in range(B if lengths is None else max(0, min(B, lengths[s]))):
            count, told = {}, set()
            for i, t in enumerate(history[s] if history is not None else []):
                if i < (prompt[s] if prompt is not None else 0):
                    told.add(t)
                else:
                    count[t] = count.get(t, 0) + 1
            if tokens is not None:
                for j in range(b + 1):
                    if j == b or masks is None or (masks[s][b] >> j) & 1:
                        t = int(tokens[s][j])
                        count[t] = count.get(t, 0) + 1
            for t in told | set(count):
                if not 0 <= t < V:
                    continue
                x = float(z[s, b, t])
                x = x / r if x > 0 else x * r
                c = count.get(t, 0)
                mag = abs(x) + abs(f * c) + abs(p)
                if c:
                    x = x - f * c - p
                z[s, b, t] = x
                # z times the rounded reciprocal: two steps; f c + p: one; the difference: one of the result
                err[s, b, t] = 4 * 2.0 ** -24 * mag if math.isfinite(mag) else 0.0
            if bias is not None:
                for t, value in dict(bias[s]).items():
                    if 0 <= t < V:
                        z[s, b, t] += value
                        x = float(z[s, b, t])
                        err[s, b, t] += 2 * 2.0 ** -24 * (abs(x) + abs(value)) if math.isfinite(x) else 0.0
            if allowed is not None and allowed[s][b] is not None:
                hide = torch.ones(V, dtype=torch.bool)
                hide[torch.tensor(sorted(t for t in allowed[s][b] if t < V), dtype=torch.long)] = False
                z[s, b, hide] = -math.inf
                err[s, b, hide] = 0
    return z, err


def pack_allowed(allowed, S, B, V, extra=0):
    """Bit words [S, B, words] of sets of tokens; bits behind the vocabulary and words behind the last are set too."""
    words = (V + 31) // 32 + extra
    out = torch.full((S, B, words), -1, dtype=torch.int32)
    for s in range(S):
        for b in range(B):
            if allowed[s][b] is None:
                continue
            bits = [0] * ((V + 31) // 32)
            for t in allowed[s][b]:
                bits[t // 32] |= 1 << (t % 32)
            if V % 32:
                bits[-1] |= (-1 << (V % 32)) & 0xFFFFFFFF
            out[s, b, :len(bits)] = torch.tensor([x - (1 << 32) if x >> 31 else x for x in bits], dtype=torch.int32)
    return out


def targets_of(z, allowed, lengths=None):
    """Largest logit of those allowed, lowest index; NaN ranks as -inf; -1 where none is allowed or not in use."""
    S, B, V = z.shape
    out = [[-1] * B for _ in range(S)]
    for s in range(S):
        for b in range(B if lengths is None else max(0, min(B, lengths[s]))):
            row = torch.nan_to_num(z[s, b], nan=-math.inf, posinf=math.inf, neginf=-math.inf)
            ids = range(V) if allowed is None or allowed[s][b] is None else sorted(t for t in allowed[s][b] if t < V)
            ids = torch.tensor(list(ids), dtype=torch.long)
            if len(ids):
                vals = row[ids]
                out[s][b] = int(ids[(vals == vals.max()).nonzero()[0, 0]])
    return out


def walk(target, tokens, masks=None, lengths=None):
    """(accepted, next_token, path) by the definition."""
    S, B = len(target), len(target[0])
    accepted, nxt, paths = [], [], []
    for s in range(S):
        used = B if lengths is None else max(0, min(B, lengths[s]))
        path = [0] if used else []
        while path:
            here, found = path[-1], None
            for c in range(here + 1, used):
                below = c and (masks[s][c] & ((1 << c) - 1) if masks is not None else 1 << (c - 1))
                if below.bit_length() - 1 == here and target[s][here] >= 0 and int(tokens[s][c]) == target[s][here]:
                    found = c
                    break
            if found is None:
                break
            path.append(found)
        accepted.append(len(path))
        nxt.append(target[s][path[-1]] if path else -1)
        paths.append(path + [-1] * (B - len(path)))
    return accepted, nxt, paths
