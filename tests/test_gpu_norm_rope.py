"""attn_qk_norm_rope and its backward against the fp64 formulas.

Bounds. Forward: one rounding to bf16, and 2^-20 of the pair's |a| + |b| for fp32
(norm: at most 24 roundings of 2^-24; sine and cosine: a few). Backward dx: one
rounding, and 2^-18 of r (|w u| + |x r| mean|w u x r|) (sums of d <= 128 terms,
at most 40 roundings). dw: one rounding, and 2^-13 of the sum of |u x r| (a chain of
at most 2^11 fp32 additions at these sizes)."""
import pytest
import torch

import transformer_scaled_dot_attn_gb300 as A
from tests import operator_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda"

CASES = [
    # B, h, h_kv, n, d, rot, sections, interleaved, first position
    (2, 4, 2, 5, 64, 64, [32], False, 0),
    (1, 1, 1, 1, 32, 32, [16], False, 0),
    (3, 5, 1, 33, 128, 128, [64], True, 1000000),
    (2, 3, 3, 130, 64, 32, [16], False, 77),
    (1, 16, 4, 257, 128, 64, [8, 12, 12], True, 5),
    (2, 2, 7, 70, 32, 16, [3, 5], False, 2000000000),
    (1, 2, 2, 19, 128, 128, [16, 24, 24], False, -40),
    (64, 16, 16, 1, 64, 64, [32], False, 4095),
    (1, 2, 1, 9, 64, 0, [0], False, 0),
    (1, 0, 3, 40, 64, 64, [32], False, 9),
    (1, 3, 0, 40, 64, 64, [32], True, 9),
    (2, 8, 8, 700, 128, 112, [56], False, 3),
]


def make(case, seed=0):
    B, h, hkv, n, d, rot, sections, inter, first = case
    q = R.bf16(B, h, n, d, seed=seed + 1) if h else None
    k = R.bf16(B, hkv, n, d, seed=seed + 2, mult=30.0) if hkv else None
    wq = (1 + 0.3 * R.bf16(d, seed=seed + 3).float()).bfloat16() if h else None
    wk = (1 + 0.3 * R.bf16(d, seed=seed + 4).float()).bfloat16() if hkv else None
    step = torch.arange(n)
    pos = torch.stack([first + step + 3 * torch.arange(B)[:, None], first // 2 + (step // 7).expand(B, n),
                       (step % 7).expand(B, n)][:len(sections)]).to(torch.int32)
    freqs = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) / max(1, rot // 2))).float()
    return q, k, wq, wk, pos, freqs


def on(t):
    return None if t is None else t.to(DEV)


def call(fn, case, q, k, wq, wk, pos, freqs, *more, **kw):
    rot, sections, inter = case[5], case[6], case[7]
    p = pos if len(sections) > 1 else pos[0]
    return fn(on(q), on(k), on(wq), on(wk), on(p.contiguous()) if rot else None, on(freqs) if rot else None,
              *more, sections=sections if rot else None, interleaved=inter, **kw)


@pytest.mark.parametrize("case", CASES)
def test_forward(case):
    q, k, wq, wk, pos, freqs = make(case)
    got = call(A.attn_qk_norm_rope, case, q, k, wq, wk, pos, freqs)
    t = R.angles(pos, freqs, case[6])
    for x, w, y in ((q, wq, got[0]), (k, wk, got[1])):
        if x is None:
            assert y is None
            continue
        ref, mag = R.norm_rope(x, w, t, case[7], 1e-6)
        err = (y.cpu().double() - ref).abs()
        assert (err <= R.HALF_BF16 * ref.abs() + 2.0 ** -20 * mag).all(), (err - R.HALF_BF16 * ref.abs()).max()


@pytest.mark.parametrize("case", CASES)
def test_backward(case):
    q, k, wq, wk, pos, freqs = make(case, 10)
    B, h, hkv, n, d = case[:5]
    gq = R.bf16(B, h, n, d, seed=21) if h else None
    gk = R.bf16(B, hkv, n, d, seed=22) if hkv else None
    got = call(A.attn_qk_norm_rope_bwd, case, q, k, wq, wk, pos, freqs, on(gq), on(gk))
    t = R.angles(pos, freqs, case[6])
    for x, w, g, dx, dw in ((q, wq, gq, got[0], got[2]), (k, wk, gk, got[1], got[3])):
        if x is None:
            assert dx is None and dw is None
            continue
        x64 = x.double().requires_grad_()
        w64 = w.double().requires_grad_()
        R.norm_rope(x64, w64, t, case[7], 1e-6)[0].backward(g.double())
        r = 1 / torch.sqrt((x.double() ** 2).mean(-1, keepdim=True) + 1e-6)
        xr = x.double() * r
        a, b = R.columns(case[5], case[7])
        u = g.double().clone()  # the upstream gradient turned back
        c, s = torch.cos(t)[:, None], torch.sin(t)[:, None]
        u[..., a], u[..., b] = g.double()[..., a] * c + g.double()[..., b] * s, \
            g.double()[..., b] * c - g.double()[..., a] * s
        um = u.abs()
        um[..., a] = um[..., b] = g.double()[..., a].abs() + g.double()[..., b].abs()
        wu = w.double().abs() * um
        mag = r * (wu + xr.abs() * (wu * xr.abs()).mean(-1, keepdim=True))
        err = (dx.cpu().double() - x64.grad).abs()
        assert (err <= R.HALF_BF16 * x64.grad.abs() + 2.0 ** -18 * mag).all()
        werr = (dw.cpu().double() - w64.grad).abs()
        assert (werr <= R.HALF_BF16 * w64.grad.abs() + 2.0 ** -13 * (um * xr.abs()).sum((0, 1, 2))).all()


def test_backward_is_the_difference_of_the_formula():
    """The gradient that the backward returns, against central differences of the fp64 forward."""
    case = (1, 2, 1, 3, 32, 32, [16], False, 5)
    q, k, wq, wk, pos, freqs = make(case, 30)
    gq, gk = R.bf16(1, 2, 3, 32, seed=41), R.bf16(1, 1, 3, 32, seed=42)
    dq, _, dwq, _ = call(A.attn_qk_norm_rope_bwd, case, q, k, wq, wk, pos, freqs, on(gq), on(gk))
    t = R.angles(pos, freqs, [16])

    def loss(x, w):
        return (R.norm_rope(x, w, t, False, 1e-6)[0] * gq.double()).sum()

    eps = 1e-5
    for idx in [(0, 0, 0, 0), (0, 1, 2, 31), (0, 0, 1, 17)]:
        e = torch.zeros_like(q, dtype=torch.float64)
        e[idx] = eps
        diff = (loss(q.double() + e, wq) - loss(q.double() - e, wq)) / (2 * eps)
        assert abs(dq.cpu()[idx].double() - diff) <= R.HALF_BF16 * abs(diff) + 1e-4
    for c in (0, 15, 31):
        e = torch.zeros(32, dtype=torch.float64)
        e[c] = eps
        diff = (loss(q.double(), wq.double() + e) - loss(q.double(), wq.double() - e)) / (2 * eps)
        assert abs(dwq.cpu()[c].double() - diff) <= R.HALF_BF16 * abs(diff) + 1e-4


def test_in_place_and_repeated():
    case = CASES[7]
    q, k, wq, wk, pos, freqs = make(case, 50)
    first = call(A.attn_qk_norm_rope, case, q, k, wq, wk, pos, freqs)
    qd, kd = on(q), on(k)
    A.attn_qk_norm_rope(qd, kd, on(wq), on(wk), on(pos[0]), on(freqs), q_out=qd, k_out=kd)
    assert torch.equal(qd, first[0]) and torch.equal(kd, first[1])
    gq, gk = on(R.bf16(*q.shape, seed=51)), on(R.bf16(*k.shape, seed=52))
    args = (on(q), on(k), on(wq), on(wk), on(pos[0]), on(freqs))
    a = A.attn_qk_norm_rope_bwd(*args, gq, gk)
    need = A.attn_qk_norm_rope_bwd_workspace_bytes(64, 16, 16, 1, 64)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)  # NaN patterns
    b = A.attn_qk_norm_rope_bwd(*args, gq, gk, dq=gq, dk=gk, workspace=ws)
    for x, y in zip(a, b):
        assert torch.equal(x, y)


def test_zero_rows_and_no_rows():
    z = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16, device=DEV)
    w = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    q, k = A.attn_qk_norm_rope(z, z, w, w)
    assert (q == 0).all() and (k == 0).all()
    e = torch.zeros(2, 3, 0, 64, dtype=torch.bfloat16, device=DEV)
    q, k = A.attn_qk_norm_rope(e, e, w, w)
    assert q.shape == e.shape
    dw = torch.full((64,), 7.0, dtype=torch.bfloat16, device=DEV)
    _, _, dwq, dwk = A.attn_qk_norm_rope_bwd(e, e, w, w, None, None, e, e, dw_q=dw)
    assert (dwq == 0).all() and (dwk == 0).all()


def test_captured_and_replayed():
    case = CASES[3]
    q, k, wq, wk, pos, freqs = make(case, 60)
    args = [on(x) for x in (q, k, wq, wk, pos[0], freqs)]
    g = [on(R.bf16(*x.shape, seed=61)) for x in (q, k)]
    want = A.attn_qk_norm_rope_bwd(*args, *g)
    outs = [torch.zeros_like(x) for x in want]
    ws = torch.empty(A.attn_qk_norm_rope_bwd_workspace_bytes(*case[:5]), dtype=torch.uint8, device=DEV)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        A.attn_qk_norm_rope_bwd(*args, *g, dq=outs[0], dk=outs[1], dw_q=outs[2], dw_k=outs[3], workspace=ws)
    for _ in range(2):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for o, x in zip(outs, want):
            assert torch.equal(o, x)
