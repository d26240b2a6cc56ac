"""What the norm + rotation, cache and tree calls refuse, before anything is launched."""
import ctypes

import pytest
import torch

import transformer_scaled_dot_attn_gb300 as A
from transformer_scaled_dot_attn_gb300 import native_build

FAKE = 0x10000  # never dereferenced
OK, BAD, UNSUP = A.ATTN_OK, A.ATTN_ERR_INVALID_ARG, A.ATTN_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    native_build.build()
    return A.load_library()


def _nr(lib, bwd=False, ptrs=None, B=2, h=4, hkv=2, n=3, d=64, rot=64, axes=1, sec=(32,), eps=1e-6, ws=1 << 20):
    ptrs = [FAKE] * (12 if bwd else 8) if ptrs is None else ptrs
    s = None if sec is None else (ctypes.c_int * len(sec))(*sec)
    if bwd:
        return lib.attn_qk_norm_rope_bwd(*ptrs, B, h, hkv, n, d, rot, axes, s, 0, eps, FAKE if ws else None, ws, None)
    return lib.attn_qk_norm_rope(*ptrs, B, h, hkv, n, d, rot, axes, s, 0, eps, None)


def test_norm_rope(lib):
    for bwd in (False, True):
        assert _nr(lib, bwd, B=-1) == BAD
        assert _nr(lib, bwd, h=-1) == BAD
        assert _nr(lib, bwd, d=48) == UNSUP
        assert _nr(lib, bwd, rot=24, sec=(12,)) == UNSUP
        assert _nr(lib, bwd, rot=80, sec=(40,)) == BAD
        assert _nr(lib, bwd, axes=4, sec=(8, 8, 8, 8)) == UNSUP
        assert _nr(lib, bwd, axes=2, sec=(8, 8)) == BAD
        assert _nr(lib, bwd, axes=2, sec=(40, -8)) == BAD
        assert _nr(lib, bwd, axes=2, sec=None) == BAD
        assert _nr(lib, bwd, eps=0.0) == BAD
        assert _nr(lib, bwd, eps=float("nan")) == BAD
        assert _nr(lib, bwd, h=65000, hkv=600) == UNSUP
        count = 12 if bwd else 8
        for i in range(count):
            ptrs = [FAKE] * count
            ptrs[i] = None
            assert _nr(lib, bwd, ptrs=ptrs) == BAD, i
            ptrs[i] = FAKE + 2
            assert _nr(lib, bwd, ptrs=ptrs) == BAD, i
    assert _nr(lib, n=0, ptrs=[None] * 8) == OK
    assert _nr(lib, True, ws=0) == BAD
    need = A.attn_qk_norm_rope_bwd_workspace_bytes(2, 4, 2, 3, 64)
    assert need > 0 and _nr(lib, True, ws=need - 1) == BAD
    assert A.attn_qk_norm_rope_bwd_workspace_bytes(2, 4, 2, 0, 64) == 0
    assert A.attn_qk_norm_rope_bwd_workspace_bytes(2, 4, 2, 3, 48) == 0


def test_cache(lib):
    def write(ptrs=None, B=2, h=2, n=3, m=10, d=64):
        return lib.attn_cache_write(*([FAKE] * 8 if ptrs is None else ptrs), B, h, n, m, d, None)

    def read(ptrs=None, B=2, h=2, m=10, d=64):
        return lib.attn_cache_read(*([FAKE] * 7 if ptrs is None else ptrs), B, h, m, d, None)

    for f in (write, read):
        assert f(B=-1) == BAD
        assert f(m=0) == BAD
        assert f(d=80) == UNSUP
        assert f(B=65536, h=65536) == UNSUP
        assert f(B=0) == OK
    assert write(n=-1) == BAD
    assert write(n=0, ptrs=[None] * 8) == OK
    for i in range(6):  # the exponent arrays come together
        ptrs = [FAKE] * 8
        ptrs[i] = None
        assert write(ptrs) == BAD
        ptrs = [FAKE] * 7
        ptrs[i] = None
        assert read(ptrs) == BAD
    for i in (0, 1, 2, 3, 6, 7):
        ptrs = [FAKE] * 8
        ptrs[i] = FAKE + 2
        assert write(ptrs) == BAD
    for i in (0, 1, 4, 5, 6):
        ptrs = [FAKE] * 7
        ptrs[i] = FAKE + 2
        assert read(ptrs) == BAD


def test_tree(lib):
    def call(ptrs=None, B=2, h=4, hkv=2, n=3, m=5000, d=64, scale=0.1, ws=FAKE, ws_bytes=1 << 30):
        return lib.attn_decode_tree(*([FAKE] * 9 if ptrs is None else ptrs), B, h, hkv, n, m, d, scale, ws, ws_bytes,
                                    None)

    assert call(n=0) == BAD
    assert call(n=65) == BAD
    assert call(m=0) == BAD
    assert call(B=-1) == BAD
    assert call(h=5) == BAD
    assert call(hkv=0) == BAD
    assert call(d=256) == UNSUP
    assert call(B=40000) == UNSUP
    assert call(h=1 << 20, hkv=2) == UNSUP
    assert call(scale=float("inf")) == BAD
    assert call(B=0, ptrs=[None] * 9) == OK
    for i in (0, 1, 2, 3, 5, 6):
        ptrs = [FAKE] * 9
        ptrs[i] = None
        assert call(ptrs) == BAD, i
    for i in (0, 1, 2, 3, 4, 7, 8):
        ptrs = [FAKE] * 9
        ptrs[i] = FAKE + 2
        assert call(ptrs) == BAD, i
    need = A.attn_decode_tree_workspace_bytes(2, 4, 2, 3, 5000, 64)
    assert need > 0
    assert call(ws=None) == BAD
    assert call(ws=FAKE + 8) == BAD
    assert call(ws_bytes=need - 1) == BAD
    assert A.attn_decode_tree_workspace_bytes(0, 4, 2, 3, 5000, 64) == 0
    assert A.attn_decode_tree_workspace_bytes(2, 4, 3, 3, 5000, 64) == 0


def test_binding_refuses_cpu_tensors(lib):
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    w = torch.ones(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        A.attn_qk_norm_rope(x, x, w, w)
    with pytest.raises(ValueError, match="CUDA"):
        A.attn_cache_write(x, x, x, x)
    with pytest.raises(ValueError, match="CUDA"):
        A.attn_decode_tree(x, x, x)
    with pytest.raises(ValueError, match="quantised"):
        A.attn_cache_read(x, x, None, None)


@pytest.mark.gpu
def test_binding_checks_tensors(lib):
    bf = dict(dtype=torch.bfloat16, device="cuda")
    q, k = torch.zeros(1, 4, 3, 64, **bf), torch.zeros(1, 2, 3, 64, **bf)
    w = torch.ones(64, **bf)
    freqs = torch.ones(32, device="cuda")
    pos = torch.zeros(1, 3, dtype=torch.int32, device="cuda")
    with pytest.raises(TypeError, match="positions"):
        A.attn_qk_norm_rope(q, k, w, w, pos.long(), freqs)
    with pytest.raises(ValueError, match="positions"):
        A.attn_qk_norm_rope(q, k, w, w, pos[:, :2].contiguous(), freqs)
    with pytest.raises(ValueError, match="sections"):
        A.attn_qk_norm_rope(q, k, w, w, pos[None].repeat(2, 1, 1), freqs)
    with pytest.raises(ValueError, match="sections"):
        A.attn_qk_norm_rope(q, k, w, w, pos[None].repeat(2, 1, 1), freqs, sections=[32])
    with pytest.raises(A.AttnError):
        A.attn_qk_norm_rope(q, k, w, w, pos[None].repeat(2, 1, 1), freqs, sections=[16, 8])
    with pytest.raises(ValueError, match="contiguous"):
        A.attn_qk_norm_rope(q.transpose(1, 2).contiguous().transpose(1, 2), k, w, w, pos, freqs)
    with pytest.raises(TypeError, match="q"):
        A.attn_qk_norm_rope(q.float(), k, w, w, pos, freqs)
    cache = torch.zeros(1, 2, 16, 64, **bf)
    e = torch.zeros(1, 2, 16, dtype=torch.uint8, device="cuda")
    f8 = cache.to(torch.float8_e4m3fn)
    with pytest.raises(TypeError, match="cache"):
        A.attn_cache_write(k, k, cache, cache, k_exp=e, v_exp=e)
    with pytest.raises(TypeError, match="v_exp"):
        A.attn_cache_write(k, k, f8, f8, k_exp=e, v_exp=None)
    with pytest.raises(ValueError, match="v_exp"):
        A.attn_cache_write(k, k, cache, cache, v_exp=e)
    with pytest.raises(ValueError, match="k has shape"):
        A.attn_cache_write(q, q, cache, cache)
    with pytest.raises(ValueError, match="kv_len"):
        A.attn_cache_write(k, k, cache, cache, torch.zeros(2, dtype=torch.int32, device="cuda"))
    with pytest.raises(A.AttnError):
        A.attn_decode_tree(torch.zeros(1, 3, 3, 64, **bf), cache, cache)  # 3 heads on 2 key heads
    with pytest.raises(A.AttnError):
        A.attn_decode_tree(torch.zeros(1, 4, 65, 64, **bf), cache, cache)
    with pytest.raises(TypeError, match="tree"):
        A.attn_decode_tree(q, cache, cache, tree=torch.zeros(1, 3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="q has shape"):
        A.attn_decode_tree(torch.zeros(1, 4, 3, 32, **bf), cache, cache)
    with pytest.raises(ValueError, match="workspace"):
        A.attn_decode_tree(q, cache, cache, workspace=torch.zeros(4))
    for call, name in ((lambda: A.attn_qk_norm_rope(q, k, w, w, None, freqs), "positions"),
                       (lambda: A.attn_qk_norm_rope(q, k, w, w, pos, 1.0), "freqs"),
                       (lambda: A.attn_qk_norm_rope(None, None, w, w), "k"),
                       (lambda: A.attn_cache_write(None, k, cache, cache), "k"),
                       (lambda: A.attn_cache_write(k, None, cache, cache), "v"),
                       (lambda: A.attn_decode_tree(None, cache, cache), "q"),
                       (lambda: A.attn_decode_tree(q, cache, None), "v cache")):
        with pytest.raises(TypeError, match=name):
            call()
    with pytest.raises(ValueError, match="dimensions"):
        A.attn_decode_tree(q[0], cache, cache)
