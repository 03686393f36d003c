"""The attention entries refuse bad arguments on the host, before anything is launched (CPU only: the
addresses below are never dereferenced)."""
import ctypes

import pytest
import torch

import linear_attention_sequence_rule_b200 as gdn

FAKE = 1 << 20
BAD, UNS, WSP = gdn.GDN_ERR_INVALID_ARGUMENT, gdn.GDN_ERR_UNSUPPORTED, gdn.GDN_ERR_WORKSPACE
NONE = ctypes.c_size_t(-1).value


def call(fn, base, kw):
    rc = fn(**(base | kw))
    assert rc != gdn.GDN_OK and fn.__name__ in gdn.gdn_last_error()
    return rc


FWD = dict(q=FAKE, k=FAKE, v=FAKE, out=FAKE, lse=None, B=1, T=64, Hq=4, Hk=2, d=64, cu_seqlens=None,
           dtype=gdn.GDN_DTYPE_BF16, scale=0.125, stream=None)
SHARED = [(dict(dtype=7), UNS), (dict(d=96), UNS), (dict(d=256), UNS), (dict(Hq=5), BAD), (dict(Hk=0), BAD),
          (dict(Hq=0), BAD), (dict(Hq=1 << 17), BAD), (dict(B=0), BAD), (dict(T=0), BAD),
          (dict(T=-1, cu_seqlens=FAKE), BAD), (dict(B=1 << 16, T=1 << 16), BAD), (dict(T=1 << 30, Hq=64), BAD),
          (dict(scale=0.0), BAD), (dict(scale=-1.0), BAD), (dict(scale=float("nan")), BAD),
          (dict(scale=float("inf")), BAD), (dict(q=None), BAD), (dict(out=None), BAD), (dict(v=FAKE + 8), BAD),
          (dict(cu_seqlens=FAKE + 4), BAD), (dict(lse=FAKE + 4), BAD),
          (dict(B=1 << 24, Hq=256, cu_seqlens=FAKE), BAD)]


@pytest.mark.parametrize("kw,code", SHARED)
def test_attn_fwd(kw, code):
    assert call(gdn.gdn_attn_fwd, FWD, kw) == code


BWD = FWD | dict(lse=FAKE, dout=FAKE, dq=FAKE, dk=FAKE, dv=FAKE, workspace=FAKE, workspace_bytes=1 << 20)


@pytest.mark.parametrize("kw,code", SHARED + [(dict(lse=None), BAD), (dict(dout=None), BAD), (dict(dk=None), BAD),
                                              (dict(dv=FAKE + 2), BAD), (dict(workspace=None), WSP),
                                              (dict(workspace_bytes=4), WSP), (dict(workspace=FAKE + 16), BAD)])
def test_attn_bwd(kw, code):
    assert call(gdn.gdn_attn_bwd, BWD, kw) == code


def test_attn_bwd_workspace():
    f = gdn.gdn_attn_bwd_workspace_bytes
    assert f(2, 100, 4, 2, 64, 0, 1) >= 2 * 100 * 4 * 4 and f(2, 100, 4, 2, 64, 1, 1) >= 100 * 4 * 4
    assert f(1, 0, 4, 2, 64, 0, 1) == NONE and f(1, 64, 3, 2, 64, 0, 1) == NONE and f(1, 64, 4, 2, 80, 0, 1) == NONE


PLAN = dict(lens=FAKE, added=FAKE, block_table=FAKE, free_list=FAKE, free_head=FAKE, cu_seqlens=FAKE, slots=FAKE,
            positions=FAKE, lens_out=FAKE, free_head_out=FAKE, status=FAKE, N=4, max_blocks=8, num_free=3, rows=9,
            page=64, stream=None)


@pytest.mark.parametrize("kw,code", [(dict(page=48), UNS), (dict(page=0), UNS), (dict(N=16385), UNS), (dict(N=0), BAD),
                                     (dict(max_blocks=0), BAD), (dict(max_blocks=1 << 25), BAD),
                                     (dict(num_free=-1), BAD), (dict(rows=-1), BAD), (dict(lens=None), BAD),
                                     (dict(slots=None), BAD), (dict(slots=FAKE + 4), BAD), (dict(free_head=FAKE + 2), BAD),
                                     (dict(status=FAKE + 1), BAD), (dict(free_list=None), BAD), (dict(status=None), BAD),
                                     (dict(block_table=FAKE + 4), BAD)])
def test_cache_plan(kw, code):
    assert call(gdn.gdn_cache_plan, PLAN, kw) == code


APP = dict(k=FAKE, v=FAKE, slots=FAKE, k_cache=FAKE, v_cache=FAKE, k_scale=FAKE, v_scale=FAKE, rows=5, Hk=2, d=128,
           page=32, num_pages=10, dtype=gdn.GDN_DTYPE_BF16, stream=None)


@pytest.mark.parametrize("kw,code", [(dict(dtype=9), UNS), (dict(d=32), UNS), (dict(page=8), UNS), (dict(rows=-1), BAD),
                                     (dict(Hk=0), BAD), (dict(num_pages=0), BAD), (dict(num_pages=1 << 26), BAD),
                                     (dict(k=None), BAD), (dict(v_scale=None), BAD), (dict(slots=FAKE + 4), BAD),
                                     (dict(k_cache=FAKE + 1), BAD)])
def test_cache_append(kw, code):
    assert call(gdn.gdn_cache_append, APP, kw) == code


DEC = dict(q=FAKE, k_cache=FAKE, v_cache=FAKE, k_scale=FAKE, v_scale=FAKE, block_table=FAKE, lens=FAKE, out=FAKE, N=2,
           Hq=8, Hk=2, d=128, page=64, num_pages=10, max_blocks=2, dtype=gdn.GDN_DTYPE_BF16, scale=0.1,
           workspace=None, workspace_bytes=0, stream=None)


@pytest.mark.parametrize("kw,code", [(dict(dtype=9), UNS), (dict(d=256), UNS), (dict(page=256), UNS), (dict(Hq=7), BAD),
                                     (dict(N=0), BAD), (dict(N=1 << 24), BAD), (dict(max_blocks=0), BAD),
                                     (dict(num_pages=0), BAD), (dict(scale=0.0), BAD), (dict(lens=None), BAD),
                                     (dict(out=FAKE + 8), BAD), (dict(max_blocks=4096), WSP)])
def test_attn_decode(kw, code):
    assert call(gdn.gdn_attn_decode, DEC, kw) == code


def test_attn_decode_workspace():
    f = gdn.gdn_attn_decode_workspace_bytes
    assert f(2, 8, 2, 128, 64, 2, 1) == 0 and f(1, 8, 2, 128, 64, 1024, 1) > 0
    assert f(0, 8, 2, 128, 64, 2, 1) == NONE and f(2, 8, 2, 128, 60, 2, 1) == NONE


def test_torch_layer_refuses_without_launching():
    q, k = torch.zeros(1, 8, 4, 64), torch.zeros(1, 8, 2, 64)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.attn_fwd(q, k, k)
    with pytest.raises(ValueError, match="dimensions"):
        gdn.attn_fwd(q[0], k, k)
    with pytest.raises(ValueError, match="dtype"):
        gdn.attn_fwd(q.half(), k.half(), k.half())
    with pytest.raises(ValueError, match="offsets"):
        gdn.attn_fwd(q[0], k[0], k[0], cu_seqlens=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="3 dimensions"):
        gdn.attn_decode(q, k, k, k, k, k, k)
    with pytest.raises(ValueError, match="CUDA"):
        gdn.cache_append(k[0], k[0], torch.zeros(8, dtype=torch.int32), k, k, k, k)
