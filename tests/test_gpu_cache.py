"""attn_cache_write and attn_cache_read: codes and exponent bytes equal the fp64
definition's (the one rounding is to the code itself), everything else stays."""
import pytest
import torch

import transformer_scaled_dot_attn_gb300 as A
from tests import operator_refs as R

pytestmark = pytest.mark.gpu
DEV = "cuda"
E4M3 = torch.float8_e4m3fn


def filled(B, h, m, d, byte=0x5a):
    return (torch.full((B, h, m, d), byte, dtype=torch.uint8, device=DEV).view(E4M3),
            torch.full((B, h, m, d), byte, dtype=torch.uint8, device=DEV).view(E4M3),
            torch.full((B, h, m), 9, dtype=torch.uint8, device=DEV), torch.full((B, h, m), 9, dtype=torch.uint8, device=DEV))


def i32(x):
    return None if x is None else torch.tensor(x, dtype=torch.int32, device=DEV)


CASES = [
    # B, h_kv, n, m, d, kv_len, new_len
    (2, 3, 1, 70, 64, [70, 5], None),
    (1, 1, 1, 1, 32, None, None),
    (3, 2, 17, 40, 128, [40, 17, 30], [17, 3, 0]),
    (2, 2, 33, 33, 32, [33, 20], [33, 20]),
    (2, 1, 10, 20, 64, [4, 20], [10, 10]),        # more new rows than the length: the first drop out
    (3, 1, 5, 12, 128, [-3, 99, 6], [9, 2, -1]),  # clamped
    (2, 2, 300, 1000, 128, [1000, 777], [300, 299]),
]


@pytest.mark.parametrize("quantised", [True, False])
@pytest.mark.parametrize("case", CASES)
def test_write(case, quantised):
    B, h, n, m, d, lens, new = case
    k = R.bf16(B, h, n, d, seed=1) * torch.exp2(R.bf16(B, h, n, 1, seed=2) * 6)
    v = R.bf16(B, h, n, d, seed=3, mult=1e-3)
    kc, vc, ke, ve = filled(B, h, m, d)
    if not quantised:
        kc, vc, ke, ve = (torch.full((B, h, m, d), 3.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)), None, None, None
        kc, vc = list(kc)
    want = [x.cpu().float() for x in (kc, vc)]
    wbytes = [None, None] if ke is None else [ke.cpu(), ve.cpu()]
    for c, x in enumerate((k, v)):
        codes, bytes_ = R.quantise(x)
        for b in range(B):
            L = m if lens is None else min(max(lens[b], 0), m)
            nn = n if new is None else min(max(new[b], 0), n)
            for i in range(nn):
                if L - nn + i >= 0:
                    want[c][b, :, L - nn + i] = codes[b, :, i].float() if quantised else x[b, :, i].float()
                    if quantised:
                        wbytes[c][b, :, L - nn + i] = bytes_[b, :, i]
    got = A.attn_cache_write(k.to(DEV), v.to(DEV), kc, vc, i32(lens), new_len=i32(new), k_exp=ke, v_exp=ve)
    assert got[0] is kc and got[1] is vc
    for x, w in zip((kc, vc), want):
        assert torch.equal(x.cpu().float(), w)
    if quantised:
        assert torch.equal(ke.cpu(), wbytes[0]) and torch.equal(ve.cpu(), wbytes[1])


def test_write_of_every_magnitude():
    """Rows whose largest value runs over every bf16 magnitude (subnormal and largest
    included), and rows of zeros, infinities and NaN."""
    mags = torch.arange(0, 0x7f80, 31, dtype=torch.int32)
    rows = torch.zeros(len(mags) + 4, 64, dtype=torch.bfloat16)
    top = mags.to(torch.int16).view(torch.bfloat16)
    g = torch.Generator().manual_seed(5)
    rows[:len(mags)] = (top[:, None].double() * (torch.rand(len(mags), 64, generator=g).double() * 2 - 1)).bfloat16()
    rows[:len(mags), 7] = top
    rows[len(mags), :] = -0.0
    rows[len(mags) + 1, :4] = torch.tensor([float("inf"), -float("inf"), 3.0, 448.0])
    rows[len(mags) + 2, :3] = torch.tensor([float("nan"), 1.0, -2.0])
    rows[len(mags) + 3, :] = float("inf")
    n = rows.shape[0]
    kc, vc, ke, ve = filled(1, 1, n, 64)
    x = rows[None, None].to(DEV)
    A.attn_cache_write(x, x, kc, vc, k_exp=ke, v_exp=ve)
    codes, bytes_ = R.quantise(rows)
    got = kc.cpu().float()[0, 0].double()
    assert torch.equal(ke.cpu()[0, 0], bytes_) and torch.equal(ve.cpu()[0, 0], bytes_)
    nan = torch.isnan(codes)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], codes[~nan])
    back, _ = A.attn_cache_read(kc, vc, ke, ve)
    back = back.cpu()[0, 0].double()
    value = codes * torch.exp2(bytes_.double() - 127)[:, None]
    assert torch.equal(torch.isnan(back), nan)
    assert torch.equal(back[~nan], value[~nan])
    # half a code step: 2^-4 of the value, or of the row's least normal code 2^-6 2^e (finite, unsaturated rows)
    ok = (top.double() <= 448 * 2.0 ** 119) & (top != 0)
    src = rows[:len(mags)].double()
    err = (back[:len(mags)] - src).abs()
    bound = 2.0 ** -4 * src.abs() + 2.0 ** -10 * torch.exp2(bytes_[:len(mags)].double() - 127)[:, None]
    assert (err[ok] <= bound[ok]).all()


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("B,h,m,lens", [(2, 3, 37, [37, 4]), (1, 1, 1, None), (3, 1, 200, [0, 300, -1]), (2, 4, 1025, [1000, 1])])
def test_read(B, h, m, d, lens):
    g = torch.Generator().manual_seed(m)
    codes = torch.randint(0, 256, (B, h, m, d), generator=g, dtype=torch.uint8)
    codes[(codes & 0x7f) == 0x7f] = 0x30
    bytes_ = torch.randint(10, 247, (B, h, m), generator=g, dtype=torch.uint8)
    for b in range(B):  # what lies behind a sequence is anyone's
        L = m if lens is None else min(max(lens[b], 0), m)
        codes[b, :, L:] = 0x7f
        bytes_[b, :, L:] = 255
    kc, vc = codes.to(DEV).view(E4M3), codes.flip(3).contiguous().to(DEV).view(E4M3)
    k, v = A.attn_cache_read(kc, vc, bytes_.to(DEV), bytes_.to(DEV), i32(lens))
    for b in range(B):
        L = m if lens is None else min(max(lens[b], 0), m)
        for got, c in ((k, codes), (v, codes.flip(3))):
            ref = c.view(E4M3).float().double()[b, :, :L] * torch.exp2(bytes_[b, :, :L].double() - 127)[..., None]
            assert torch.equal(got.cpu()[b, :, :L].double(), ref)
            assert (got[b, :, L:] == 0).all()


def test_far_offsets():
    """A cache of more than 2^32 codes: rows of the last head."""
    B, h, m, d = 1, 34, 1 << 20, 128
    kc = torch.zeros(B, h, m, d, dtype=torch.uint8, device=DEV).view(E4M3)
    vc = torch.zeros(B, h, m, d, dtype=torch.uint8, device=DEV).view(E4M3)
    ke = torch.full((B, h, m), 127, dtype=torch.uint8, device=DEV)
    ve = ke.clone()
    k, v = R.bf16(B, h, 3, d, seed=8), R.bf16(B, h, 3, d, seed=9)
    A.attn_cache_write(k.to(DEV), v.to(DEV), kc, vc, k_exp=ke, v_exp=ve)
    for x, c, e in ((k, kc, ke), (v, vc, ve)):
        codes, bytes_ = R.quantise(x)
        assert torch.equal(c[:, :, -3:].cpu().float().double(), codes) and torch.equal(e[:, :, -3:].cpu(), bytes_)
        assert int(c.view(torch.uint8)[:, -1, :-3].count_nonzero()) == 0
    o, lse = A.attn_decode_tree(k.to(DEV), kc, vc, i32([m]), k_exp=ke, v_exp=ve)
    # the zero keys have score 0 and zero values; only the last three positions carry a value
    for hd in (0, h - 1):
        kk = kc[0, hd, -3:].cpu().double() * torch.exp2(ke[0, hd, -3:].cpu().double() - 127)[:, None]
        vv = vc[0, hd, -3:].cpu().double() * torch.exp2(ve[0, hd, -3:].cpu().double() - 127)[:, None]
        for i in range(3):
            w = torch.exp((kk[:i + 1] @ k[0, hd, i].double()) / d ** 0.5)
            total = (m - 3) + w.sum()
            ref = (w @ vv[:i + 1]) / total
            assert abs(lse[0, hd, i].item() - torch.log(total).item()) <= 2.0 ** -14
            assert ((o[0, hd, i].cpu().double() - ref).abs() <= 2.0 ** -6 * (w @ vv[:i + 1].abs()) / total).all()


@pytest.mark.parametrize("rows", [1, 40, 200])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_every_code_as_a_value(d, rows):
    """A step that sees one position returns that position's value row: every finite code,
    at small, ordinary and large exponents, through each of the tree step's kernels."""
    codes = torch.arange(256, dtype=torch.uint8)
    codes = codes[(codes & 0x7f) != 0x7f]
    codes = torch.cat([codes, codes[:2 * d - len(codes) % d - (d if len(codes) % d == 0 else 0)]])
    codes = codes[:len(codes) // d * d].reshape(-1, d)
    for byte in (127 - 117, 100, 127, 135, 136, 246):
        B = codes.shape[0]
        n = min(rows, 64)
        h = (rows + n - 1) // n
        kc = torch.zeros(B, 1, n, d, dtype=torch.uint8)
        vc = kc.clone()
        vc[:, 0, 0] = codes
        e = torch.full((B, 1, n), byte, dtype=torch.uint8)
        q = R.bf16(B, h, n, d, seed=3)
        tree = torch.ones(B, n, dtype=torch.int64)  # every query sees position 0 alone
        o, _ = A.attn_decode_tree(q.to(DEV), kc.to(DEV).view(E4M3), vc.to(DEV).view(E4M3), tree=tree.to(DEV),
                                  k_exp=e.to(DEV), v_exp=e.to(DEV))
        want = codes.view(E4M3).float().double() * 2.0 ** (byte - 127)
        assert torch.equal(o.cpu().double(), want[:, None, None].expand(B, h, n, d))


def test_captured_and_replayed():
    B, h, n, m, d = 2, 2, 3, 40, 64
    k, v = R.bf16(B, h, n, d, seed=1).to(DEV), R.bf16(B, h, n, d, seed=2).to(DEV)
    kc, vc, ke, ve = filled(B, h, m, d, 0)
    lens = i32([10, 40])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        A.attn_cache_write(k, v, kc, vc, lens, k_exp=ke, v_exp=ve)
    for step in (0, 3):
        lens.copy_(i32([10 + step, 40 - step]))
        graph.replay()
        back, _ = A.attn_cache_read(kc, vc, ke, ve, lens)
        codes, bytes_ = R.quantise(k.cpu())
        value = codes * torch.exp2(bytes_.double() - 127)[..., None]
        assert torch.equal(back[0, :, 7 + step:10 + step].cpu().double(), value[0])
        assert torch.equal(back[1, :, 37 - step:40 - step].cpu().double(), value[1])
