"""fp64 forms of the norm + rotation, the quantised cache and the tree step, for the tests."""
import math

import torch

F64 = torch.float64
HALF_BF16 = torch.finfo(torch.bfloat16).eps / 2  # a rounding's largest relative error
U32 = torch.finfo(torch.float32).eps / 2


def bf16(*shape, seed, mult=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * mult).bfloat16()


# ---------------------------------------------------------------- norm + rotation

def angles(pos, freqs, sections):
    """fp64 angles [B, n, pairs] of positions [axes, B, n]."""
    out, at = [], 0
    for axis, size in enumerate(sections):
        out.append(pos[axis].to(F64)[..., None] * freqs[at:at + size].to(F64))
        at += size
    return torch.cat(out, -1) if out else torch.zeros(*pos.shape[1:], 0, dtype=F64)


def columns(rot, interleaved):
    i = torch.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def norm_rope(x, w, t, interleaved, eps):
    """(result, |a| + |b| of each column's pair) of x [B, h, n, d] at angles t [B, n, pairs]."""
    x, w = x.to(F64), w.to(F64)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    a, b = columns(2 * t.shape[-1], interleaved)
    c, s = torch.cos(t)[:, None], torch.sin(t)[:, None]
    z, mag = y.clone(), y.abs()
    z[..., a], z[..., b] = y[..., a] * c - y[..., b] * s, y[..., a] * s + y[..., b] * c
    mag[..., a] = mag[..., b] = y[..., a].abs() + y[..., b].abs()
    return z, mag


# ---------------------------------------------------------------- quantised rows

def quantise(x):
    """(values of the codes, exponent bytes) of the rows of bf16 x, in fp64."""
    x = x.to(F64)
    fin = torch.where(torch.isfinite(x), x.abs(), 0.0)
    top = fin.amax(-1)
    e = torch.zeros(top.shape, dtype=torch.int64)
    for k in range(-117, 120):  # the least exponent that holds the row; 119 where none does
        e = torch.where((top > 448 * 2.0 ** k) & (top > 0), min(k + 1, 119), e) if k > -117 else \
            torch.where(top > 448 * 2.0 ** k, k + 1, torch.where(top > 0, -117, 0))
    z = torch.clamp(x * torch.exp2(-e.to(F64))[..., None], -448, 448)
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(z / step) * step, (e + 127).to(torch.uint8)


# ---------------------------------------------------------------- tree attention

def random_tree(B, n, seed):
    """Mask words [B][n] of random trees: each token hangs on an earlier one or on the text."""
    g = torch.Generator().manual_seed(seed)
    words = []
    for _ in range(B):
        row = []
        for i in range(n):
            parent = int(torch.randint(-1, i, (1,), generator=g)) if i else -1
            row.append((1 << i) | (row[parent] if parent >= 0 else 0))
        words.append(row)
    return words


def words_tensor(words):
    return torch.tensor([[x - (1 << 64) if x >> 63 else x for x in r] for r in words], dtype=torch.int64)


def visible(n, L, words):
    """[n, L]: the cached positions each of the n newest sees."""
    see = torch.zeros(n, L, dtype=torch.bool)
    see[:, :max(0, L - n)] = True
    for i in range(n):
        for t in range(max(0, n - L), n):
            see[i, L - n + t] = bool(words[i] >> t & 1) if words is not None else t <= i
    return see


def tree_step(q, k, v, lens, words, scale):
    """fp64 (O, lse, A = sum_j p_j |v_j|, S = largest scale sum_c |q_c k_c|) of q [B, h, n, d] over k, v
    [B, h_kv, m, d] (real values, any dtype). Positions that a query does not see take no part."""
    B, h, n, d = q.shape
    group = h // k.shape[1]
    o = torch.zeros(B, h, n, d, dtype=F64)
    A, lse, S = o.clone(), torch.full((B, h, n), -math.inf, dtype=F64), torch.zeros(B, h, n, dtype=F64)
    for b in range(B):
        L = lens[b]
        if L == 0:
            continue
        see = visible(n, L, None if words is None else words[b])
        for hd in range(h):
            kk, vv, qq = k[b, hd // group, :L].to(F64), v[b, hd // group, :L].to(F64), q[b, hd].to(F64)
            x = torch.where(see, scale * (qq @ kk.T), -math.inf)
            lse[b, hd] = torch.logsumexp(x, -1)
            p = torch.where(see, torch.exp(x - lse[b, hd, :, None]), 0.0)
            o[b, hd], A[b, hd] = p @ vv, p @ vv.abs()
            S[b, hd] = torch.where(see, abs(scale) * (qq.abs() @ kk.abs().T), 0.0).amax(-1)
    return o, lse, A, S


def check_tree(got_o, got_lse, ref):
    """O: its rounding to bf16, the weights' rounding to bf16 (relative, so at most
    HALF_BF16 sum p|v|) and 2^-14 sum p|v| for the fp32 scores and sums. lse: fp32
    scores, accumulated over d <= 128 products with at most 2^-23 each of their
    magnitude, i.e. 2^-16 S, and as much again of 1 for the exponentials and logs."""
    o, lse, A, S = ref
    got_o, got_lse = got_o.cpu().to(F64), got_lse.cpu().to(F64)
    empty = torch.isneginf(lse)
    assert torch.equal(torch.isneginf(got_lse), empty)
    assert (got_o[empty] == 0).all()
    err = (got_o - o).abs() - (HALF_BF16 * o.abs() + (HALF_BF16 + 2.0 ** -14) * A)
    assert err.max() <= 0, f"O off by {err.max():.3e} more than allowed at {torch.argmax(err)}"
    off = torch.where(empty, 0.0, (got_lse - lse).abs() - 2.0 ** -16 * (1 + S))
    assert off.nan_to_num(posinf=1.0).max() <= 0, f"lse off by {off.max():.3e} more than allowed"
