"""attn_decode_tree against the fp64 step (tests/operator_refs.py holds the bounds)."""
import pytest
import torch

import transformer_scaled_dot_attn_gb300 as A
from seeded_inputs import DECODE_WORKLOADS
from tests import operator_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)


def caches(B, hkv, m, d, quantised, seed):
    """(call's k, v, exponent bytes on the GPU; the values they hold)."""
    k, v = R.bf16(B, hkv, m, d, seed=seed), R.bf16(B, hkv, m, d, seed=seed + 1)
    if not quantised:
        return (k.to(DEV), v.to(DEV), None, None), (k, v)
    # rows of different magnitude: the values' scales spread over eight binades
    v = (v.float() * torch.exp2(torch.randint(-4, 5, (B, hkv, m, 1), generator=torch.Generator().manual_seed(seed)).float())).bfloat16()
    (kc, ke), (vc, ve) = R.quantise(k), R.quantise(v)
    vals = [c * torch.exp2(e.double() - 127)[..., None] for c, e in ((kc, ke), (vc, ve))]
    return (kc.float().to(E4M3).to(DEV), vc.float().to(E4M3).to(DEV), ke.to(DEV), ve.to(DEV)), vals


def run(q, c, lens, words, scale, **kw):
    o, lse = A.attn_decode_tree(q.to(DEV), c[0], c[1], i32(lens), None if words is None else R.words_tensor(words).to(DEV),
                                k_exp=c[2], v_exp=c[3], scale=scale, **kw)
    assert A.attn_get_device_status() == A.ATTN_OK
    return o, lse


CASES = [
    # B, h, h_kv, n, m, d, kv_len, tree, scale multiplier
    (2, 2, 2, 1, 100, 64, None, False, 1.0),
    (1, 1, 1, 1, 1, 32, None, False, 1.0),
    (2, 4, 2, 5, 333, 128, [333, 40], True, 1.0),
    (3, 7, 1, 3, 200, 64, [200, 3, 1], True, 1.0),       # 21 rows: a second row block; fewer cached than drafted
    (2, 2, 1, 64, 700, 64, [700, 64], True, 1.0),
    (1, 8, 1, 64, 513, 128, None, True, 1.0),            # 512 rows
    (2, 4, 4, 16, 257, 32, [0, 257], True, 1.0),         # an empty cache
    (2, 6, 2, 9, 90, 32, [90, 31], False, -0.7),
    (1, 3, 3, 17, 65, 128, [40], True, 0.0),
    (4, 4, 1, 33, 2100, 128, [2100, 1024, 63, 1999], True, 1.0),
    (2, 32, 4, 20, 1500, 64, [1500, 900], True, 2.0),
    (1, 2, 2, 2, 9000, 128, None, False, 1.0),           # a long cache split over many CTAs
    (1, 40, 1, 4, 777, 32, [700], True, 1.0),
    # hundreds of parts to join for few heads
    (1, 8, 1, 1, 40011, 128, [39000], False, 1.0),
    (1, 2, 2, 1, 60000, 32, None, False, 1.0),
    (1, 1, 1, 64, 25000, 64, [24987], True, 1.0),
    (1, 5, 1, 60, 30000, 64, None, True, 1.0),
    (2, 16, 2, 64, 20000, 128, [20000, 7], True, 1.0),
]


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_matches_the_definition(case, quantised):
    B, h, hkv, n, m, d, lens, tree, mult = case
    q = R.bf16(B, h, n, d, seed=7)
    c, (k, v) = caches(B, hkv, m, d, quantised, 11)
    words = R.random_tree(B, n, 3) if tree else None
    scale = mult / d ** 0.5
    o, lse = run(q, c, lens, words, scale)
    R.check_tree(o, lse, R.tree_step(q, k, v, lens or [m] * B, words, scale))


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("n,group,d", [(64, 8, 128), (64, 1, 128), (8, 1, 128), (64, 4, 64), (33, 1, 32), (16, 1, 64)])
def test_long_caches(n, group, d, quantised):
    """Hundreds of key tiles through every ring, many times, in batches of different lengths."""
    B, hkv, m = 3, 4, 20011
    q = R.bf16(B, hkv * group, n, d, seed=7)
    c, (k, v) = caches(B, hkv, m, d, quantised, 11)
    words = R.random_tree(B, n, 3)
    lens = [20011, 5000, 17777]
    for _ in range(20):
        o, lse = run(q, c, lens, words, d ** -0.5)
    for b, g in ((0, 0), (1, 2), (2, 3)):
        hs = slice(g * group, (g + 1) * group)
        ref = R.tree_step(q[b:b + 1, hs], k[b:b + 1, g:g + 1], v[b:b + 1, g:g + 1], [lens[b]], [words[b]], d ** -0.5)
        R.check_tree(o[b:b + 1, hs], lse[b:b + 1, hs], ref)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 15, 16, 17, 31, 32, 33, 48, 63, 64])
def test_every_row_count(n):
    """Rows around the tiles' edges, lengths around the key tiles' edges."""
    for quantised, d, group in ((False, 64, 1), (True, 128, 3)):
        lens = [n, 127 + n, 129, 256]
        q = R.bf16(4, group, n, d, seed=n)
        c, (k, v) = caches(4, 1, 260, d, quantised, n + 100)
        words = R.random_tree(4, n, n)
        o, lse = run(q, c, lens, words, d ** -0.5)
        R.check_tree(o, lse, R.tree_step(q, k, v, lens, words, d ** -0.5))


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("n,group,d,hkv,m", [
    (6, 1, 64, 1, 150), (40, 4, 128, 1, 150), (64, 1, 32, 1, 150),
    # batches large enough for tiles of 128 query rows, pairs of them, pairs of two
    (64, 2, 32, 32, 2300), (40, 4, 128, 24, 1200), (64, 8, 64, 8, 1100), (64, 8, 128, 8, 1100)])
def test_what_a_query_does_not_see_never_reaches_it(n, group, d, hkv, m, quantised):
    """NaN and infinities behind the sequence and in drafted positions: queries that see them
    get NaN or infinities, the others the finite result; words of 0 are rows that see the
    text alone, or nothing."""
    B, lens = 3, [m - 30, m - 50, n]
    q = R.bf16(B, hkv * group, n, d, seed=1)
    c, (k, v) = caches(B, hkv, m, d, quantised, 5)
    words = R.random_tree(B, n, 9)
    words[0][n - 1] = words[2][n - 1] = words[2][0] = 0
    for b in range(B):
        if quantised:
            c[0].view(torch.uint8)[b, :, lens[b]:] = 0x7f
            c[1].view(torch.uint8)[b, :, lens[b]:] = 0xff
            c[2][b, :, lens[b]:] = 255
            c[3][b, :, lens[b]:] = 255
        else:
            c[0][b, :, lens[b]:] = float("nan")
            c[1][b, :, lens[b]:] = float("inf")
    bad = [1, 3]  # drafted tokens whose key (the first) and value (the second) are not finite
    for b in range(B):
        if quantised:
            c[0].view(torch.uint8)[b, :, lens[b] - n + bad[0], d // 2] = 0x7f
            c[1].view(torch.uint8)[b, :, lens[b] - n + bad[1], 3] = 0x7f
        else:
            c[0][b, :, lens[b] - n + bad[0], d // 2] = float("nan")
            c[1][b, :, lens[b] - n + bad[1], 3] = float("inf")
    o, lse = run(q, c, lens, words, d ** -0.5)
    ref = list(R.tree_step(q, k, v, lens, words, d ** -0.5))
    hit = torch.tensor([[[bool(w >> bad[0] & 1) for w in r]] * (hkv * group) for r in words])
    val = torch.tensor([[[bool(w >> bad[1] & 1) for w in r]] * (hkv * group) for r in words])
    o, lse = o.cpu(), lse.cpu()
    assert torch.isnan(o[hit]).all() and torch.isnan(lse[hit]).all()
    col = o[..., 3]
    assert not torch.isfinite(col[val]).any()
    clean = ~hit & ~val
    assert clean.any() and torch.isfinite(o[clean]).all()
    only = ~hit & val  # of these rows only the value's own column is touched
    keep = torch.arange(d) != 3
    assert torch.isfinite(o[only][:, keep]).all()
    sel = ~hit
    o2, ref_o = o.clone(), ref[0].clone()
    o2[..., 3] = torch.where(val, 0.0, o2[..., 3].float()).bfloat16()
    ref_o[..., 3] = torch.where(val, 0.0, ref_o[..., 3])
    R.check_tree(o2[sel], lse[sel], [x[sel] for x in (ref_o, ref[1], ref[2], ref[3])])


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("n", [17, 31, 33, 48, 63, 64])
def test_row_counts_in_large_batches(n, d):
    """Rows around the edges of large query tiles, lengths around the key tiles' edges."""
    B, hkv, m = 16, 8, 1600
    lens = [n, 127 + n, 129, 256, 1600, 1599, 1025, 0, 1, 128, 1537, 1000, 1600, 640, 641, 639]
    words = R.random_tree(B, n, n)
    for quantised, group in ((False, 1), (True, 3), (False, 5), (True, 8)):
        q = R.bf16(B, hkv * group, n, d, seed=n)
        c, (k, v) = caches(B, hkv, m, d, quantised, n + 100)
        o, lse = run(q, c, lens, words, d ** -0.5)
        for b in range(B):
            g = b % hkv
            hs = slice(g * group, (g + 1) * group)
            ref = R.tree_step(q[b:b + 1, hs], k[b:b + 1, g:g + 1], v[b:b + 1, g:g + 1], [lens[b]], [words[b]], d ** -0.5)
            R.check_tree(o[b:b + 1, hs], lse[b:b + 1, hs], ref)


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("n,group", [(64, 1), (40, 4), (64, 8)])
def test_short_sequences_of_many_scales(n, group, d, quantised):
    """A thousand (sequence, head)s of one or two key tiles, which differ in scale by up to 2^24:
    nothing of one may be taken for another's. Some hold a NaN value that some of their
    queries see."""
    B, hkv, m, most = 128, 8, 3500, 170
    g = torch.Generator().manual_seed(n + d)
    lens = [64 + int(torch.randint(0, 100, (1,), generator=g)) for _ in range(B)]
    q = R.bf16(B, hkv * group, n, d, seed=n)
    k, v = R.bf16(B, hkv, most, d, seed=1), R.bf16(B, hkv, most, d, seed=2)
    k, v = ((x.float() * torch.exp2(torch.randint(lo, hi, (B, hkv, 1, 1), generator=g).float())).bfloat16()
            for x, lo, hi in ((k, -12, 1), (v, -12, 13)))
    words = R.random_tree(B, n, n)
    bad = torch.rand(B, hkv, generator=g) < 0.3

    def cache(x):
        c = torch.zeros(B, hkv, m, *x.shape[3:], dtype=torch.uint8 if quantised else torch.bfloat16, device=DEV)
        c[:, :, :most] = x.to(DEV)
        return c

    if quantised:
        (kc, ke), (vc, ve) = R.quantise(k), R.quantise(v)
        c = [cache(x.float().to(E4M3).view(torch.uint8)) for x in (kc, vc)] + [cache(ke), cache(ve)]
        k, v = (x * torch.exp2(e.double() - 127)[..., None] for x, e in ((kc, ke), (vc, ve)))
    else:
        c = [cache(k), cache(v), None, None]
    for b in range(B):
        for h in range(hkv):
            if bad[b, h]:
                c[1][b, h, lens[b] - n + 5, 7] = 0x7f if quantised else float("nan")
    if quantised:
        c[:2] = [x.view(E4M3) for x in c[:2]]
    o, lse = run(q, c, lens, words, d ** -0.5)
    o, lse = o.cpu(), lse.cpu()
    nan = torch.isnan(o)
    sees5 = torch.tensor([[bool(w >> 5 & 1) for w in r] for r in words])
    assert torch.equal(nan[..., 7], (sees5[:, None] & bad[..., None]).repeat_interleave(group, 1))
    assert not nan[..., torch.arange(d) != 7].any()
    for b in range(B):
        h = b % hkv
        hs = slice(h * group, (h + 1) * group)
        ref = list(R.tree_step(q[b:b + 1, hs], k[b:b + 1, h:h + 1], v[b:b + 1, h:h + 1], [lens[b]], [words[b]], d ** -0.5))
        got = o[b:b + 1, hs].clone()
        got[nan[b:b + 1, hs]] = 0
        ref[0][nan[b:b + 1, hs]] = 0
        R.check_tree(got, lse[b:b + 1, hs], ref)


@pytest.mark.parametrize("quantised", [False, True])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_grow_along_the_cache(d, quantised):
    """A running maximum that has to move many times: keys longer from tile to tile, and back."""
    B, hkv, group, n, m = 4, 8, 8, 40, 2000
    q = R.bf16(B, hkv * group, n, d, seed=1)
    c, (k, v) = caches(B, hkv, m, d, False, 3)
    size = (1 + 40 * torch.sin(torch.arange(m) / 300.0).abs())[:, None]
    k = (k.float() * size).bfloat16()
    if quantised:
        (kc, ke), (vc, ve) = R.quantise(k), R.quantise(v)
        k, v = (x * torch.exp2(e.double() - 127)[..., None] for x, e in ((kc, ke), (vc, ve)))
        c = (kc.float().to(E4M3).to(DEV), vc.float().to(E4M3).to(DEV), ke.to(DEV), ve.to(DEV))
    else:
        c = (k.to(DEV), v.to(DEV), None, None)
    o, lse = run(q, c, None, None, d ** -0.5)
    for b in range(B):
        hs = slice(b * group, (b + 1) * group)
        ref = R.tree_step(q[b:b + 1, hs], k[b:b + 1, b:b + 1], v[b:b + 1, b:b + 1], [m], None, d ** -0.5)
        R.check_tree(o[b:b + 1, hs], lse[b:b + 1, hs], ref)


def test_causal_words_equal_no_words_and_plain_decoding():
    B, h, n, m, d = 2, 4, 4, 500, 64
    q = R.bf16(B, h, n, d, seed=1)
    c, _ = caches(B, h, m, d, False, 2)
    lens = [500, 123]
    a = run(q, c, lens, None, d ** -0.5)
    b = run(q, c, lens, [[(2 << i) - 1 for i in range(n)]] * B, d ** -0.5)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    o, lse = A.attn_decode(q.to(DEV), c[0], c[1], i32(lens))
    # two roundings of the weights' sums apart
    assert (a[1] - lse).abs().max() <= 2.0 ** -14
    assert (a[0].float() - o.float()).abs().max() <= 2.0 ** -6 * c[1].float().abs().max()


@pytest.mark.parametrize("quantised", [False, True])
def test_same_bits_from_any_workspace_and_stream(quantised):
    B, h, hkv, n, m, d = 2, 4, 2, 20, 3000, 128
    q = R.bf16(B, h, n, d, seed=1)
    c, _ = caches(B, hkv, m, d, quantised, 2)
    words = R.random_tree(B, n, 4)
    first = run(q, c, [3000, 1500], words, 0.1)
    ws = torch.full((A.attn_decode_tree_workspace_bytes(B, h, hkv, n, m, d),), 255, dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    again = run(q, c, [3000, 1500], words, 0.1, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_allocations_belong_to_the_stream_of_the_call():
    """What a call on another stream allocates is not handed out again on this one while the
    call is still waiting to run."""
    B, h, hkv, n, m, d = 2, 4, 2, 20, 3000, 128
    q = R.bf16(B, h, n, d, seed=1).to(DEV)
    c, _ = caches(B, hkv, m, d, False, 2)
    first = A.attn_decode_tree(q, c[0], c[1], scale=0.1)
    busy = torch.ones(8192, 8192, device=DEV)
    need = A.attn_decode_tree_workspace_bytes(B, h, hkv, n, m, d)
    assert need > 0
    side = torch.cuda.Stream()
    for _ in range(5):
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            for _ in range(4):
                busy @ busy
        again = A.attn_decode_tree(q, c[0], c[1], scale=0.1, stream=side)
        junk = [torch.full((need,), 255, dtype=torch.uint8, device=DEV) for _ in range(4)]
        torch.cuda.synchronize()
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
        assert all(bool((x == 255).all()) for x in junk)
        del junk, again


def test_captured_step_follows_the_lengths():
    B, h, hkv, n, m, d = 2, 4, 2, 3, 600, 64
    q = R.bf16(B, h, n, d, seed=1)
    c, (k, v) = caches(B, hkv, m, d, True, 2)
    lens, qd = i32([10, 20]), q.to(DEV)
    ws = torch.empty(max(16, A.attn_decode_tree_workspace_bytes(B, h, hkv, n, m, d)), dtype=torch.uint8, device=DEV)
    o, lse = torch.empty_like(qd), torch.empty(B, h, n, device=DEV)
    A.attn_decode_tree(qd, c[0], c[1], lens, k_exp=c[2], v_exp=c[3], out=o, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        A.attn_decode_tree(qd, c[0], c[1], lens, k_exp=c[2], v_exp=c[3], out=o, lse=lse, workspace=ws)
    for new in ([600, 1], [0, 333]):
        lens.copy_(i32(new))
        graph.replay()
        torch.cuda.synchronize()
        R.check_tree(o, lse, R.tree_step(q, k, v, new, None, d ** -0.5))


@pytest.mark.parametrize("quantised", [False, True])
def test_captured_layers_among_copies_and_another_stream(quantised):
    """A step of several layers in one graph: lengths copied in, norm and rotation, cache write,
    tree attention into the next layer's input, a cache read on another stream that joins again.
    Replays with new inputs give the bits of eager calls."""
    layers, B, h, hkv, n, m, d = 3, 2, 8, 2, 6, 1500, 64
    g = torch.Generator(device=DEV).manual_seed(1)
    dtype = E4M3 if quantised else torch.bfloat16
    kc, vc = ([torch.zeros(B, hkv, m, d, dtype=torch.float32, device=DEV).to(dtype) for _ in range(layers)] for _ in range(2))
    ke, ve = ([torch.full((B, hkv, m), 127, dtype=torch.uint8, device=DEV) if quantised else None for _ in range(layers)]
              for _ in range(2))
    w = torch.ones(d, device=DEV).bfloat16()
    freqs = (10000.0 ** (-torch.arange(d // 2, device=DEV) / (d // 2))).float()
    kv = [torch.randn(B, hkv, n, d, device=DEV, generator=g).bfloat16() for _ in range(2 * layers)]
    x, given, pos = torch.zeros(B, h, n, d, device=DEV).bfloat16(), i32([n, n]), i32([list(range(n))] * B)
    lens = torch.zeros_like(given)
    ws = torch.empty(max(16, A.attn_decode_tree_workspace_bytes(B, h, hkv, n, m, d)), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()

    def step():
        lens.copy_(given)
        q = x
        for i in range(layers):
            qn, kn = A.attn_qk_norm_rope(q, kv[2 * i], w, w, pos, freqs)
            A.attn_cache_write(kn, kv[2 * i + 1], kc[i], vc[i], lens, k_exp=ke[i], v_exp=ve[i])
            back = None
            if quantised:
                side.wait_stream(torch.cuda.current_stream())
                back = A.attn_cache_read(kc[i], vc[i], ke[i], ve[i], lens, stream=side)
            q, lse = A.attn_decode_tree(qn, kc[i], vc[i], lens, k_exp=ke[i], v_exp=ve[i], workspace=ws)
            if quantised:
                torch.cuda.current_stream().wait_stream(side)
        return q, lse, back

    def start(seed, at):
        gen = torch.Generator(device=DEV).manual_seed(seed)
        x.copy_(torch.randn(B, h, n, d, device=DEV, generator=gen))
        given.copy_(i32(at))
        for c in kc + vc:
            c.copy_((0.1 * torch.randn(B, hkv, m, d, device=DEV, generator=gen)).to(dtype))

    start(1, [n, n])
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed, at in ((2, [1500, 40]), (3, [7, 1111]), (4, [600, 1499])):
        start(seed, at)
        for _ in range(3):
            graph.replay()
        torch.cuda.synchronize()
        mine = [t.clone() for t in got[:2]] + [t.clone() for t in got[2] or ()]
        start(seed, at)
        want = step()
        torch.cuda.synchronize()
        for a, b in zip(mine, list(want[:2]) + list(want[2] or ())):
            assert torch.equal(a, b)
    assert A.attn_get_device_status() == A.ATTN_OK


@pytest.mark.parametrize("name", list(DECODE_WORKLOADS))
def test_benchmark_steps_quantised(name):
    """The benchmark's decoding steps at full size over quantised caches, four heads of each checked."""
    B, h, n, m, d = DECODE_WORKLOADS[name]
    g = torch.Generator(device=DEV).manual_seed(3)
    q, k, v = (torch.randn(B, h, s, d, device=DEV, generator=g).bfloat16() for s in (n, m, m))
    kc, vc = (torch.empty(B, h, m, d, dtype=E4M3, device=DEV) for _ in range(2))
    ke, ve = (torch.empty(B, h, m, dtype=torch.uint8, device=DEV) for _ in range(2))
    A.attn_cache_write(k, v, kc, vc, k_exp=ke, v_exp=ve)
    k, v = A.attn_cache_read(kc, vc, ke, ve, k=k, v=v)
    o, lse = A.attn_decode_tree(q, kc, vc, k_exp=ke, v_exp=ve)
    assert A.attn_get_device_status() == A.ATTN_OK
    for b, hd in ((0, 0), (B // 2, 3), (B - 1, h - 1)):
        s = (slice(b, b + 1), slice(hd, hd + 1))
        R.check_tree(o[s], lse[s], R.tree_step(q[s].cpu(), k[s].cpu(), v[s].cpu(), [m], None, d ** -0.5))


def test_a_step_from_projection_to_output():
    """The operators as a program chains them: projection, norm and rotation, cache write,
    tree attention over the quantised cache; the prompt's part read back for attn_fwd."""
    B, h, d, dm, prompt, n, m = 2, 4, 64, 256, 75, 9, 128
    hd = h * d
    w_qkv = R.bf16(dm, 3 * hd, seed=1, mult=dm ** -0.5).to(DEV)
    wq, wk = ((1 + 0.2 * R.bf16(d, seed=s).float()).bfloat16().to(DEV) for s in (2, 3))
    freqs = (10000.0 ** (-torch.arange(d // 2, dtype=torch.float64) / (d // 2))).float().to(DEV)
    kc, vc = (torch.zeros(B, h, m, d, dtype=torch.uint8, device=DEV).view(E4M3) for _ in range(2))
    ke, ve = (torch.full((B, h, m), 127, dtype=torch.uint8, device=DEV) for _ in range(2))
    real = [75, 50]

    def step(x, pos, lens, new):
        q, k, v = A.attn_qkv_projection(x, x, w_qkv, h, d)
        q, k = A.attn_qk_norm_rope(q, k, wq, wk, pos.to(torch.int32).to(DEV).contiguous(), freqs, q_out=q, k_out=k)
        A.attn_cache_write(k, v, kc, vc, i32(lens), new_len=i32(new), k_exp=ke, v_exp=ve)
        return q, k, v

    x0 = R.bf16(B, prompt, dm, seed=4).to(DEV)
    q0, k0, v0 = step(x0, torch.arange(prompt).expand(B, prompt), real, real)
    # the prompt through the forward, from the cache as it is held
    kr, vr = A.attn_cache_read(kc, vc, ke, ve, i32(real))
    o0, _ = A.attn_fwd(q0, kr, vr, causal=True, kv_len=i32(real))
    assert torch.isfinite(o0).all()
    words = R.random_tree(B, n, 8)
    depth = torch.tensor([[bin(w).count("1") - 1 for w in r] for r in words])
    x1 = R.bf16(B, n, dm, seed=5).to(DEV)
    lens = [L + n for L in real]
    q1, k1, v1 = step(x1, depth + torch.tensor(real)[:, None], lens, [n] * B)
    o1, lse1 = A.attn_decode_tree(q1, kc, vc, i32(lens), R.words_tensor(words).to(DEV), k_exp=ke, v_exp=ve)
    kr, vr = A.attn_cache_read(kc, vc, ke, ve, i32(lens))
    R.check_tree(o1, lse1, R.tree_step(q1.cpu(), kr.cpu(), vr.cpu(), lens, words, d ** -0.5))
    # what the cache holds are the rows that were written, to half a code step
    for b in range(B):
        rows = torch.cat([k0[b, :, :real[b]], k1[b]], 1).double()
        err = (kr[b, :, :lens[b]].double() - rows).abs()
        top = rows.abs().amax(-1, keepdim=True)
        assert (err <= 2.0 ** -4 * rows.abs() + 2.0 ** -17 * top).all()
    y = A.attn_out_projection(o1, R.bf16(hd, dm, seed=6, mult=hd ** -0.5).to(DEV))
    assert torch.isfinite(y).all() and A.attn_get_device_status() == A.ATTN_OK
