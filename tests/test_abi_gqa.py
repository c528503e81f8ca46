"""Refusals of the grouped-query attention and page-pool entry points: decided
on the host before anything is launched (no GPU needed)."""
import ctypes

import pytest
import torch

from sparse_attention_logits_b200 import _build

import sparse_attention_logits_b200 as dsa

INVALID, UNSUPPORTED = 1, 2
vp = ctypes.c_void_p
FAKE = vp(0x1000)           # never dereferenced: validation fails first
ODD = vp(0x1008)


@pytest.fixture(scope="module")
def lib():
    _build.build_library()
    return dsa._lib


def test_append_refusals(lib):
    def f(k=FAKE, ld=1024, dt=1, n=4, table=FAKE, batch=2, width=4, page=16, pages=8, hkv=8, d=128, kc=FAKE, kv=1, ks=None,
          vs=None, rb=FAKE):
        return lib.kv_cache_append(k, ld, FAKE, 1024, dt, rb, FAKE, n, table, batch, width, page, pages, hkv, d, kc, FAKE, kv,
                                   ks, vs, None)
    assert f(n=0) == 0 and f(n=-1) == INVALID
    assert f(k=None) == INVALID and f(k=ODD) == INVALID and f(table=None) == INVALID and f(rb=None) == INVALID
    assert f(ld=1023) == INVALID and f(ld=1028) == INVALID              # rows overlap; rows not 16-byte aligned
    assert f(kc=ODD) == INVALID
    assert f(kv=2) == INVALID and f(kv=2, ks=FAKE) == INVALID           # fp8 without (both) scales
    assert f(kv=1, ks=FAKE, vs=FAKE) == INVALID
    assert f(kv=3) == UNSUPPORTED and f(dt=2) == UNSUPPORTED and f(dt=1, kv=0) == UNSUPPORTED
    assert f(d=96) == UNSUPPORTED and f(d=256) == UNSUPPORTED
    for bad in ("batch", "width", "page", "pages", "hkv", "d"):
        assert f(**{bad: 0}) == INVALID
    assert f(pages=1 << 30, page=16) == UNSUPPORTED
    assert f(batch=1 << 20, width=1 << 20) == UNSUPPORTED


def test_decode_refusals(lib):
    def f(q=FAKE, ld=4096, dt=1, kv=1, ks=None, vs=None, rows=3, h=32, hkv=8, d=128, scale=0.1, out=FAKE, ws=vp(0x10000),
          wsb=1 << 40, page=16, width=4):
        return lib.gqa_decode_attention(q, ld, dt, FAKE, FAKE, kv, ks, vs, FAKE, 2, width, page, 100, FAKE, FAKE, rows, h, hkv, d,
                                        scale, out, FAKE, ws, wsb, None)
    assert f(rows=0) == 0 and f(rows=-1) == INVALID
    assert f(q=None) == INVALID and f(q=ODD) == INVALID and f(ld=4095) == INVALID and f(out=ODD) == INVALID
    assert f(h=33) == INVALID and f(h=0) == INVALID
    assert f(scale=0.0) == INVALID and f(scale=float("nan")) == INVALID and f(scale=float("inf")) == INVALID
    assert f(dt=0, kv=1, ld=8192) == UNSUPPORTED and f(dt=1, kv=0) == UNSUPPORTED and f(dt=2) == UNSUPPORTED
    assert f(kv=2) == INVALID
    assert f(d=32) == UNSUPPORTED
    assert f(rows=1 << 30, width=1 << 10) == UNSUPPORTED


def test_prompt_refusals(lib):
    def f(q=FAKE, ldq=4096, ldk=1024, dt=1, cu=FAKE, n=3, total=100, h=32, hkv=8, d=128, scale=0.1, out=FAKE):
        return lib.gqa_prompt_attention(q, ldq, FAKE, ldk, FAKE, 1024, dt, cu, n, total, h, hkv, d, scale, out, FAKE,
                                        vp(0x10000), 1 << 40, None)
    assert f(n=0) == 0 and f(total=0) == 0 and f(n=-1) == INVALID and f(total=-1) == INVALID
    assert f(q=None) == INVALID and f(cu=None) == INVALID and f(out=None) == INVALID
    assert f(q=ODD) == INVALID and f(ldq=4095) == INVALID and f(ldk=1020) == INVALID and f(ldk=1028) == INVALID
    assert f(h=33) == INVALID and f(hkv=0) == INVALID
    assert f(dt=2) == UNSUPPORTED and f(d=192) == UNSUPPORTED
    assert f(scale=-1.0) == INVALID
    assert f(total=2 ** 31 - 1, h=4096, ldq=4096 * 128) == UNSUPPORTED


def test_pool_refusals(lib):
    def ext(table=FAKE, batch=4, width=8, page=16, n=2, pages=100, seqs=FAKE):
        return lib.kv_pages_extend(table, batch, width, page, FAKE, FAKE, pages, seqs, FAKE, n, None)
    assert ext(n=0) == 0
    assert ext(table=None) == INVALID and ext(seqs=None) == INVALID and ext(n=-1) == INVALID
    for bad in ("batch", "width", "page", "pages"):
        assert ext(**{bad: 0}) == INVALID
    assert ext(n=4097) == UNSUPPORTED and ext(pages=(1 << 22) + 1) == UNSUPPORTED
    assert ext(batch=1 << 16, width=1 << 16) == UNSUPPORTED
    assert lib.kv_pages_free(FAKE, 4, 8, 16, FAKE, FAKE, 100, None, 2, None) == INVALID

    def caches(ptrs, sizes):
        return (vp * len(ptrs))(*ptrs), (ctypes.c_size_t * len(sizes))(*sizes), len(ptrs)

    def fork(c, ws=FAKE, wsb=1 << 20, n=2):
        return lib.kv_pages_fork(FAKE, 4, 8, 16, FAKE, FAKE, 100, FAKE, FAKE, n, *c, ws, wsb, None)
    good = caches([0x1000], [4096])
    assert fork(good, n=0) == 0
    assert fork(good, ws=None) == INVALID and fork(good, wsb=8) == INVALID and fork(good, ws=vp(0x1004)) == INVALID
    assert fork(caches([0x1008], [4096])) == INVALID and fork(caches([None], [4096])) == INVALID
    assert fork(caches([0x1000], [24])) == UNSUPPORTED and fork(caches([0x1000], [0])) == UNSUPPORTED
    assert lib.kv_pages_copy(*good, 100, None, FAKE, 2, None) == INVALID
    assert lib.kv_pages_copy(*good, 0, FAKE, FAKE, 2, None) == INVALID
    assert lib.kv_pages_copy(*good, 100, FAKE, FAKE, 0, None) == 0

    def compact(t_out=vp(0x100000), r_out=vp(0x200000), wsb=1 << 20):
        return lib.kv_pages_compact(vp(0x1000), 4, 8, vp(0x8000), 100, *good, t_out, r_out, FAKE, wsb, None)
    assert compact(t_out=None) == INVALID and compact(wsb=100) == INVALID
    assert compact(t_out=vp(0x1004)) == INVALID and compact(r_out=vp(0x8010)) == INVALID        # overlap without being the input


def test_workspace_sizes(lib):
    assert lib.kv_pages_fork_workspace_size(10) >= 80 and lib.kv_pages_fork_workspace_size(0) == 0
    assert lib.kv_pages_compact_workspace_size(1000) >= 16 * 1000
    assert lib.gqa_decode_attention_workspace_size(0, 8, 2, 128, 1) == 0
    assert lib.gqa_decode_attention_workspace_size(4, 9, 2, 128, 1) == 0
    a, b = (lib.gqa_decode_attention_workspace_size(r, 32, 8, 128, 1) for r in (1, 1000))
    assert 0 < a < b


def test_binding_refuses_cpu_tensors_and_wrong_types():
    t = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        dsa.kv_pages_free(t, t[:, 0].contiguous(), t[0], t[0], 16)
    with pytest.raises(ValueError):
        dsa.gqa_prompt_attention(torch.zeros(4, 2, 64), torch.zeros(4, 2, 64), torch.zeros(4, 2, 64),
                                 torch.tensor([0, 4], dtype=torch.int32), 0.1)
