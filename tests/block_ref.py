"""Plain implementations in 64 bits of the product with packed weights and of
the attention, with bounds on what a float32 computation of them may be off.

Bounds.  A float32 sum of n terms, in any order, is off by at most n 2^-24
times the sum of the terms' magnitudes (each of at most n - 1 additions rounds
a partial sum that is below that).  A rounding to a type of eps = finfo.eps is
off by at most eps / 2 of the value (and by half the smallest subnormal).
"""
import numpy as np
import torch

U = 2.0 ** -24
KINDS = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


def half_step(kind):
    return torch.finfo(kind).eps / 2


def least(kind):
    """Half the smallest subnormal (0 where it is below anything that counts)."""
    return 2.0 ** -25 if kind == torch.float16 else 0.0


# ---------------------------------------------------------------------------
# packed weights
# ---------------------------------------------------------------------------
def pack(codes, bits):
    """Rows as little-endian bit streams in int32 words."""
    rows, cols = codes.shape
    words = max((cols * bits + 31) // 32, 1)
    stream = np.zeros((rows, words * 32), dtype=np.uint8)
    for b in range(bits):
        stream[:, b:cols * bits:bits] = (codes >> b) & 1
    return np.packbits(stream, axis=1, bitorder="little").view("<u4").view(np.int32).reshape(rows, words)


def difference(codes, zeros, group):
    """q - z, float64."""
    per = group or max(codes.shape[1], 1)
    return codes.astype(np.float64) - np.repeat(zeros, per, axis=1)[:, :codes.shape[1]]


def weights(codes, scales, zeros, group):
    per = group or max(codes.shape[1], 1)
    return difference(codes, zeros, group) * np.repeat(scales.astype(np.float64), per, axis=1)[:, :codes.shape[1]]


def activated(v, act):
    """(value, bound on the derivative)"""
    if act == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v), 1.0
    if act == "silu":
        return v * torch.sigmoid(v), 1.1
    if act == "gelu":
        return 0.5 * v * torch.erfc(-v * 2.0 ** -0.5), 1.13
    return v, 1.0


def product(x, w, bias, act, residual, out_kind):
    """(y, bound) of ``act(x w^T + bias) + residual``; x [n, d] and w [m, d]
    float64.  The sums: one addition a product, and one for a group's part."""
    y = x @ w.t()
    size = x.abs() @ w.t().abs()
    if bias is not None:
        y, size = y + bias, size + bias.abs()
    off = (x.shape[1] * 17 / 16 + 4) * U * size
    y, slope = activated(y, act)
    # float32 exp and erf, a division and two products: a few units of the value
    off = slope * off + (16 * U * size if act in ("silu", "gelu") else 0.0)
    if residual is not None:
        off = off + U * (y.abs() + residual.abs())
        y = y + residual
    return y, off + half_step(out_kind) * (y.abs() + off) + least(out_kind)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
def attend(q, k, v, keep, scale, kind):
    """(y, bound) of one head: q [n, d], k and v [m, d] float64, keep [n, m].
    Rows that keep nothing are zero."""
    k = torch.where(keep.any(0)[:, None], k, torch.zeros_like(k))
    v = torch.where(keep.any(0)[:, None], v, torch.zeros_like(v))
    n, d = q.shape
    y, off = torch.zeros(n, d, dtype=torch.float64), torch.zeros(n, d, dtype=torch.float64)
    for i in range(n):
        seen = keep[i]
        if not bool(seen.any()):
            continue
        ki, vi = k[seen], v[seen]
        s = ki @ q[i] * scale
        size = (ki.abs() @ q[i].abs()).max() * scale
        p = torch.exp(s - s.max())
        l = p.sum()
        y[i] = p @ vi / l
        # a score: d products, the scale, the maximum's subtraction and the exponent's rounding;
        # a weight is off by that much of itself, and twice, since the sum is too
        score = (d + 4) * U * size + 4 * U * (s.max() - s.min()) + 8 * U
        spread = p @ vi.abs() / l
        many = seen.sum() * U
        off[i] = (2 * score + 2 * many + half_step(kind)) * spread + least(kind) * vi.abs().sum(0) / l
    return y, off + half_step(kind) * (y.abs() + off) + least(kind)


def prompts(q, k, v, starts, causal, scale, kind):
    """(y, bound, touched rows) over packed sequences; q [n, h, d], k, v [n, g, d] of any type."""
    n, heads, d = q.shape
    group = heads // k.shape[1]
    y, off = torch.zeros(n, heads, d, dtype=torch.float64), torch.zeros(n, heads, d, dtype=torch.float64)
    touched = torch.zeros(n, dtype=torch.bool)
    for a, b in zip(starts[:-1], starts[1:]):
        touched[a:b] = True
        keep = torch.ones(b - a, b - a, dtype=torch.bool)
        keep = keep.tril() if causal else keep
        for h in range(heads):
            y[a:b, h], off[a:b, h] = attend(q[a:b, h].double(), k[a:b, h // group].double(),
                                            v[a:b, h // group].double(), keep, scale, kind)
    return y, off, touched


def cached(q, keys, values, table, lengths, scale, kind):
    """(y, bound) over pages; a page number outside the cache counts as masked."""
    count, heads, d = q.shape
    pages, kv, page, _ = keys.shape
    y, off = torch.zeros(count, heads, d, dtype=torch.float64), torch.zeros(count, heads, d, dtype=torch.float64)
    for b in range(count):
        length = min(max(int(lengths[b]), 0), table.shape[1] * page)
        at = [(int(table[b, j // page]), j % page) for j in range(length)]
        at = [(p, r) for p, r in at if 0 <= p < pages]
        if not at:
            continue
        p, r = torch.tensor([a[0] for a in at]), torch.tensor([a[1] for a in at])
        keep = torch.ones(1, len(at), dtype=torch.bool)
        for h in range(heads):
            g = h // (heads // kv)
            one = attend(q[b, h:h + 1].double(), keys[p, g, r].double(), values[p, g, r].double(), keep, scale, kind)
            y[b, h], off[b, h] = one[0][0], one[1][0]
    return y, off


def near(got, want, off, what=""):
    """got within off of want, NaN and infinities in the same places."""
    got = got.double().cpu()
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), f"{what}: NaN at other places"
    assert torch.equal(got[odd & ~torch.isnan(want)], want[odd & ~torch.isnan(want)]), f"{what}: infinities"
    far = torch.where(odd, torch.zeros_like(want), (got - want).abs() - off)
    worst = int(far.argmax()) if far.numel() else 0
    assert far.numel() == 0 or float(far.max()) <= 0, (
        f"{what}: {int((far > 0).sum())} of {far.numel()} off, worst at {worst}: "
        f"{got.flatten()[worst]} for {want.flatten()[worst]} (bound {off.flatten()[worst]})")


# name, tokens, rows, columns, group: products with packed weights that reach each kernel of a whole device
PACKED_KERNELS = [("few tokens", 3, 1000, 512, 128), ("few tokens", 15, 515, 1000, 0), ("few tokens", 32, 2000, 384, 64),
                  ("32 x 64", 530, 301, 384, 128), ("32 x 64", 300, 700, 1000, 0), ("32 x 64", 250, 1100, 640, 32),
                  ("64 x 128", 1100, 1035, 512, 128), ("64 x 128", 777, 1363, 1000, 0), ("64 x 128", 2700, 2801, 192, 48),
                  ("128 x 384", 2700, 2801, 384, 128), ("128 x 384", 2945, 2689, 264, 0), ("128 x 384", 4000, 2305, 512, 256)]
