"""The paged cache operators on the host: refusals (every one is decided before a device is
looked at, so made-up addresses are never touched), workspace sizes, and the tests' 64-bit
reference against torch's own attention."""
import ctypes
import math

import pytest
import torch

from hybrid_attention_ssm_b200 import build as hbuild
from hybrid_attention_ssm_b200 import hymba as H
from tests import paged_ref as R

A = 1 << 20      # an aligned address that nothing reads


@pytest.fixture(scope="module", autouse=True)
def _lib():
    hbuild.build()
    H.lib()


def cache(**kw):
    d = dict(dtype=H.DT_F16, n_pages=8, page_size=16, n_kv_heads=2, head_dim=64, page_stride=2048, head_stride=1024,
             row_stride=64, k=A, v=A, k_lo=A, k_hi=A)
    d.update(kw)
    return H.PagedKV(**d)


def table(**kw):
    d = dict(pages=A, batch=3, width=4, stride=4)
    d.update(kw)
    return H.PageTable(**d)


def append(kv=None, tb=None, **kw):
    a = dict(start=A, cu=A, n=3, src=H.DT_F32, k=A, ks=128, v=A, vs=128, q=A, qs=256, hq=4, q_out=A, base=1e4, ws=A,
             wsb=256)
    a.update(kw)
    return H.lib().hymba_paged_append(ctypes.byref(kv or cache()), ctypes.byref(tb or table()), a["start"], a["cu"],
                                      a["n"], a["src"], a["k"], a["ks"], a["v"], a["vs"], a["q"], a["qs"], a["hq"],
                                      a["q_out"], a["base"], a["ws"], a["wsb"], None)


def select(kv=None, tb=None, **kw):
    a = dict(lens=A, q=A, qs=256, hq=4, first=1, last=1, top=3, idx=A, ws=A, wsb=1 << 30)
    a.update(kw)
    return H.lib().hymba_paged_select(ctypes.byref(kv or cache()), ctypes.byref(tb or table()), a["lens"], a["q"],
                                      a["qs"], a["hq"], a["first"], a["last"], a["top"], a["idx"], a["ws"], a["wsb"],
                                      None)


def attention(kv=None, tb=None, **kw):
    a = dict(lens=A, q=A, qs=256, hq=4, scale=0.125, meta=0, window=0, idx=None, top=0, out=A + 4096, odt=H.DT_F32, os=256,
             lse=None, ws=A, wsb=1 << 30)
    a.update(kw)
    return H.lib().hymba_paged_attention(ctypes.byref(kv or cache()), ctypes.byref(tb or table()), a["lens"], a["q"],
                                         a["qs"], a["hq"], a["scale"], a["meta"], a["window"], a["idx"], a["top"],
                                         a["out"], a["odt"], a["os"], a["lse"], a["ws"], a["wsb"], None)


BAD_CACHE = [(dict(dtype=H.DT_F32), H.ERR_UNSUPPORTED), (dict(head_dim=96), H.ERR_UNSUPPORTED),
             (dict(page_size=8), H.ERR_UNSUPPORTED), (dict(page_size=48), H.ERR_UNSUPPORTED),
             (dict(page_size=512), H.ERR_UNSUPPORTED), (dict(n_pages=0), H.ERR_INVALID_ARG),
             (dict(n_kv_heads=0), H.ERR_INVALID_ARG), (dict(k_lo=None), H.ERR_INVALID_ARG),
             (dict(k_hi=A + 8), H.ERR_INVALID_ARG)]
BAD_POOL = [dict(k=None), dict(v=A + 8), dict(row_stride=60), dict(row_stride=32), dict(head_stride=1028),
            dict(page_stride=0), dict(head_stride=1000, row_stride=64), dict(page_stride=1 << 40)]
BAD_TABLE = [dict(pages=None), dict(pages=A + 2), dict(batch=0), dict(width=0), dict(stride=3)]


@pytest.mark.parametrize("call", [append, select, attention])
def test_caches_and_tables_are_checked(call):
    for kw, code in BAD_CACHE:
        assert call(kv=cache(**kw)) == code, kw
    if call is not select:                      # selection reads the bounds only
        for kw in BAD_POOL:
            assert call(kv=cache(**kw)) == H.ERR_INVALID_ARG, kw
    for kw in BAD_TABLE:
        assert call(tb=table(**kw)) == H.ERR_INVALID_ARG, kw
    assert call(ws=None) == call(ws=A + 16) == H.ERR_INVALID_ARG
    assert call(wsb=255) == H.ERR_WORKSPACE


@pytest.mark.parametrize("kw,code", [
    (dict(start=None), H.ERR_INVALID_ARG), (dict(start=A + 1), H.ERR_INVALID_ARG), (dict(cu=A + 2), H.ERR_INVALID_ARG),
    (dict(n=-1), H.ERR_INVALID_ARG), (dict(cu=None, n=2), H.ERR_INVALID_ARG), (dict(src=9), H.ERR_UNSUPPORTED),
    (dict(k=None), H.ERR_INVALID_ARG), (dict(v=None), H.ERR_INVALID_ARG), (dict(q=None), H.ERR_INVALID_ARG),
    (dict(q_out=None), H.ERR_INVALID_ARG), (dict(k=None, v=None, q=None, q_out=None), H.ERR_INVALID_ARG),
    (dict(base=-1.0), H.ERR_INVALID_ARG), (dict(base=math.nan), H.ERR_INVALID_ARG),
    (dict(base=math.inf), H.ERR_INVALID_ARG), (dict(hq=5), H.ERR_UNSUPPORTED), (dict(hq=0), H.ERR_UNSUPPORTED),
    (dict(hq=34), H.ERR_UNSUPPORTED), (dict(k=A + 4), H.ERR_INVALID_ARG), (dict(ks=64), H.ERR_INVALID_ARG),
    (dict(vs=130), H.ERR_INVALID_ARG), (dict(qs=252), H.ERR_INVALID_ARG), (dict(src=H.DT_BF16, ks=132), H.ERR_INVALID_ARG),
    (dict(q_out=A + 8), H.ERR_INVALID_ARG)])
def test_append_refusals(kw, code):
    assert append(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(lens=None), H.ERR_INVALID_ARG), (dict(q=None), H.ERR_INVALID_ARG), (dict(qs=248), H.ERR_INVALID_ARG),
    (dict(idx=None), H.ERR_INVALID_ARG), (dict(hq=3), H.ERR_UNSUPPORTED), (dict(top=0), H.ERR_INVALID_ARG),
    (dict(first=-1), H.ERR_INVALID_ARG), (dict(last=-1), H.ERR_INVALID_ARG), (dict(first=2, last=2), H.ERR_INVALID_ARG),
    (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), H.ERR_INVALID_ARG),
    (dict(kv=cache(k_lo=None, k_hi=None)), H.ERR_INVALID_ARG),
    (dict(tb=table(width=16385, stride=16385)), H.ERR_UNSUPPORTED), (dict(wsb=128), H.ERR_WORKSPACE)])
def test_select_refusals(kw, code):
    assert select(**kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(lens=A + 2), H.ERR_INVALID_ARG), (dict(q=A + 8), H.ERR_INVALID_ARG), (dict(qs=260), H.ERR_INVALID_ARG),
    (dict(hq=7), H.ERR_UNSUPPORTED), (dict(scale=math.nan), H.ERR_INVALID_ARG), (dict(scale=math.inf), H.ERR_INVALID_ARG),
    (dict(meta=-1), H.ERR_INVALID_ARG), (dict(meta=3), H.ERR_INVALID_ARG), (dict(window=-1), H.ERR_INVALID_ARG),
    (dict(idx=A, top=0), H.ERR_INVALID_ARG), (dict(idx=A, top=2, window=5), H.ERR_INVALID_ARG),
    (dict(out=None), H.ERR_INVALID_ARG), (dict(out=A), H.ERR_INVALID_ARG), (dict(out=A + 8), H.ERR_INVALID_ARG), (dict(odt=3), H.ERR_UNSUPPORTED),
    (dict(os=255), H.ERR_INVALID_ARG), (dict(lse=A + 1), H.ERR_INVALID_ARG), (dict(wsb=4096), H.ERR_WORKSPACE)])
def test_attention_refusals(kw, code):
    assert attention(**kw) == code


def test_workspace_size_grows_with_what_needs_it():
    n = ctypes.c_size_t()

    def size(batch, hq, pages, **kw):
        assert H.lib().hymba_paged_workspace_size(ctypes.byref(cache(**kw)), batch, hq, pages, ctypes.byref(n)) == H.OK
        return n.value

    a = size(1, 4, 1)
    assert a % 256 == 0 and a >= 148 * 2 * 2 * 68 * 4
    assert size(1, 4, 1, head_dim=128) > a and size(1, 32, 1) > a
    assert size(64, 4, 16384) == a     # neither the batch nor the lengths matter
    for kw, args in ((dict(), (0, 4, 1)), (dict(), (1, 5, 1)), (dict(), (1, 4, 0)), (dict(page_size=20), (1, 4, 1))):
        assert H.lib().hymba_paged_workspace_size(ctypes.byref(cache(**kw)), *args, ctypes.byref(n)) != H.OK


def test_reference_equals_library_attention():
    lens = [5, 33, 64]
    k, v, table_ = R.make_pool(lens, 16, 2, 64, torch.float16, seed=1)
    q = torch.randn(3, 6, 64, dtype=torch.float64).half()
    out, lse, _ = R.attention(k, v, table_, lens, q, 0.125)
    for b, n in enumerate(lens):
        pos = torch.arange(n)
        pg = table_[b].long()[pos // 16]
        kk, vv = (t[pg, :, pos % 16].double().transpose(0, 1).repeat_interleave(3, 0) for t in (k, v))
        want = torch.nn.functional.scaled_dot_product_attention(q[b, :, None].double(), kk, vv, scale=0.125)[:, 0]
        assert (out[b] - want).abs().max() < 1e-12
    # rotation: an angle of a quarter turn swaps the halves, and norms stay
    x = torch.randn(1, 1, 64, dtype=torch.float64)
    r = R.rotate(x, [7], 10000.0)
    assert (r.norm() - x.norm()).abs() < 1e-12
    assert torch.allclose(R.rotate(r, [-7], 10000.0), x)
    # the score is the largest value over the box's corners
    lo, hi = torch.tensor([[[-1.0, 2.0]]]), torch.tensor([[[3.0, 4.0]]])
    q2 = torch.tensor([[1.0, -1.0], [-2.0, 0.5]])
    assert R.scores(lo, hi, torch.tensor([0]), q2).item() == (3 - 2) + (2 + 2)
    assert R.select([1.0, 5.0, 5.0, 0.0, 9.0], 1, 0, 3) == [0, 1, 4]
