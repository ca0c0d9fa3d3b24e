"""The paged cache operators on the GPU against the 64-bit definitions in paged_ref.

Bounds, derived from the arithmetic (u16 = eps / 2 of the type, u = 2^-24):
  append     the angle is a phase modulo 2^64 (2^-32 of a turn when it is used), its sine and
             cosine come from fp32 polynomials (at most 4 u each), two products and a sum:
             8 u (|x1| + |x2|) and one rounding to the pool's type (u16 |ref|, 2^-25 in
             fp16's subnormals)
  attention  scores: D products in fp32 accumulation, each step off by at most 2 u of the
             running size S = scale sum|q k|, then the scale and the subtraction of the maximum:
             d = (2 D + 8) u S in the exponent's argument, for numerator and denominator alike;
             ex2.approx 4 u; the probability as two 16-bit parts u16^2 (fp16: of 2^15 p, so 2^-40
             absolute on top, below u for p > 2^-16 and added up at most n 2^-40; bf16 has a
             third part);
             the sums over n keys in at most n + 64 steps of 2 u.  Relative to max|v|:
             c = 2 d + 2 (n + 64) u + 8 u + u16^2 + 2^-24, and the output's rounding u_out |ref|
"""
import math

import pytest
import torch

from hybrid_attention_ssm_b200 import hymba as H
from tests import paged_ref as R

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.lib()


def half_step(dt):
    return torch.finfo(dt).eps / 2


def workspace(cache, B, Hq, width):
    return H.alloc_workspace(H.paged_workspace_size(cache, B, Hq, width))


def run_attention(k, v, table, lens, q, out_dtype=torch.float32, page_idx=None, lse=True, scale=None, **kw):
    cache = H.PagedCache(R.to_gpu(k), R.to_gpu(v))
    B, Hq, D = q.shape
    ws = workspace(cache, B, Hq, table.shape[1])
    out = torch.full((B, Hq, D), math.nan, dtype=out_dtype, device="cuda")
    ls = torch.full((B, Hq), math.nan, device="cuda") if lse else None
    H.paged_attention(cache, q.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), out, ws,
                      page_idx=None if page_idx is None else page_idx.cuda(), lse=ls, scale=scale, **kw)
    torch.cuda.synchronize()
    return out.cpu(), None if ls is None else ls.cpu(), H.status_read(ws)


def check_attention(got, lse, ref, v, n_max, dt, out_dt, D):
    out, rl, size = ref
    d = (2 * D + 8) * U * size[..., None]
    c = 2 * d + (2 * (n_max + 64) + 8) * U + half_step(dt) ** 2 + U
    vmax = torch.nan_to_num(v.double()).abs().max()
    bound = c * vmax + half_step(out_dt) * out.abs() + (2.0 ** -25 if out_dt == torch.float16 else 0)
    assert torch.isfinite(got.double()).all()
    err = (got.double() - out).abs()
    assert (err <= bound).all(), f"worst {float((err / bound).max()):.3f} of the bound"
    if lse is not None:
        lb = d[..., 0] + (2 * (n_max + 64) + 8) * U + 4 * U * rl.abs().nan_to_num(posinf=0)
        empty = torch.isinf(rl)
        assert torch.equal(torch.isinf(lse), empty) and (lse[empty] < 0).all()
        assert ((lse.double() - rl).abs()[~empty] <= lb[~empty]).all()


ATT = [  # Hq, Hkv, D, page, dtype, layout
    (25, 5, 64, 64, torch.float16, "page_head_row"),
    (25, 5, 64, 16, torch.bfloat16, "page_row_head"),
    (4, 2, 64, 32, torch.float16, "head_page_row"),
    (6, 6, 64, 128, torch.bfloat16, "page_head_row"),
    (16, 1, 64, 64, torch.float16, "page_row_head"),
    (32, 4, 128, 16, torch.bfloat16, "page_head_row"),
    (9, 1, 128, 32, torch.float16, "page_head_row"),
    (16, 2, 128, 256, torch.float16, "page_row_head"),
    (32, 2, 128, 64, torch.bfloat16, "head_page_row"),
]


@pytest.mark.parametrize("Hq,Hkv,D,ps,dt,layout", ATT)
def test_attention_all_positions(Hq, Hkv, D, ps, dt, layout):
    lens = [0, 1, 15, 16, 17, 63, 64, 65, ps - 1, ps, ps + 1, 200, 0, 129]
    k, v, table = R.make_pool(lens, ps, Hkv, D, dt, seed=1, layout=layout)
    q = (torch.randn(len(lens), Hq, D, generator=torch.Generator().manual_seed(2)) * 1.5).to(dt)
    ref = R.attention(k, v, table, lens, q, D ** -0.5)
    for out_dt in (torch.float32, torch.float16, torch.bfloat16):
        got, lse, status = run_attention(k, v, table, lens, q, out_dt)
        assert status == H.OK
        check_attention(got, lse, ref, v, max(lens), dt, out_dt, D)
        assert (got[0] == 0).all() and (got[12] == 0).all()


@pytest.mark.parametrize("M,W", [(0, 1), (0, 64), (8, 1), (8, 33), (128, 64), (130, 100), (300, 5), (5, 10 ** 9)])
@pytest.mark.parametrize("ps", [16, 64, 128])
def test_attention_window_and_meta(M, W, ps):
    lens = [0, 1, 7, 8, 9, 64, 100, 138, 139, 257, 500]
    Hq, Hkv, D, dt = 10, 2, 64, torch.float16
    k, v, table = R.make_pool(lens, ps, Hkv, D, dt, seed=3)
    q = torch.randn(len(lens), Hq, D, generator=torch.Generator().manual_seed(4)).to(dt)
    # pages wholly hidden may have been given back: their entries are out of the pool
    for b, n in enumerate(lens):
        seen = {p // ps for p in R.positions(n, ps, M, W)}
        for j in range(-(-n // ps)):
            if j not in seen:
                table[b, j] = -7
    ref = R.attention(k, v, table, lens, q, D ** -0.5, M, W)
    got, lse, status = run_attention(k, v, table, lens, q, n_meta=M, window=W)
    assert status == H.OK
    check_attention(got, lse, ref, v, max(lens), dt, torch.float32, D)


def test_hidden_positions_have_no_influence():
    """Positions outside the window hold infinities, the type's lowest value and NaN."""
    lens, ps, Hq, Hkv, D, dt = [300, 90], 32, 5, 1, 64, torch.float16
    k, v, table = R.make_pool(lens, ps, Hkv, D, dt, seed=5)
    q = torch.randn(2, Hq, D, generator=torch.Generator().manual_seed(6)).to(dt)
    ref = R.attention(k, v, table, lens, q, 0.125, 10, 40)
    for bad in (math.inf, -math.inf, math.nan, torch.finfo(dt).min):
        for b, n in enumerate(lens):
            for p in range(10, n - 40):
                k[table[b, p // ps], :, p % ps] = bad
                v[table[b, p // ps], :, p % ps] = bad
        got, lse, status = run_attention(k, v, table, lens, q, n_meta=10, window=40)
        assert status == H.OK
        check_attention(got, lse, ref, torch.where(v.isfinite() & (v.abs() < 100), v, 0), 300, dt, torch.float32, D)


def test_visible_nan_and_infinite_keys():
    """A visible NaN makes its rows NaN; a key of score -inf gets no weight; only such keys: NaN
    as in the formula."""
    dt, ps = torch.float16, 16
    k, v, table = R.make_pool([40, 40, 40], ps, 1, 64, dt, seed=7)
    q = torch.zeros(3, 2, 64, dtype=dt)
    q[:, :, 0] = 1.0
    k[table[0, 1].long(), 0, 3, 5] = math.nan
    k[table[1, 2].long(), 0, 1, 0] = -math.inf
    q[1, :, 1:] = 1.0
    k[table[1, 2].long(), 0, 1, 1:] = 0.0
    got, lse, _ = run_attention(k, v, table, [40, 40, 40], q)
    assert got[0].isnan().all() and lse[0].isnan().all()
    kk = k[table[1].long()].clone()
    keep = [p for p in range(40) if p != 33]
    rows = k[table[1].long()[torch.tensor(keep) // ps], 0, torch.tensor(keep) % ps].double()
    vals = v[table[1].long()[torch.tensor(keep) // ps], 0, torch.tensor(keep) % ps].double()
    want = torch.softmax(q[1].double() @ rows.T * 0.125, -1) @ vals
    # the module's bound at S < 16, max|v| < 4: 2 (2 * 64 + 8) 16 u * 4 = 1.04e-3
    assert (got[1].double() - want).abs().max() < 1.04e-3
    assert torch.isfinite(got[2]).all()


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_visible_value_that_is_not_finite(dt, bad):
    """Its channel in the heads of its group is not finite either; all else is as without it."""
    lens, ps, Hq, Hkv, D = [40, 90], 16, 6, 2, 64
    k, v, table = R.make_pool(lens, ps, Hkv, D, dt, seed=33)
    q = torch.randn(2, Hq, D, generator=torch.Generator().manual_seed(34)).to(dt)
    want, wl, _ = run_attention(k, v, table, lens, q)
    v[table[1, 2].long(), 1, 5, 7] = bad
    got, lse, status = run_attention(k, v, table, lens, q)
    assert status == H.OK and torch.equal(lse, wl)
    assert not got[1, 3:, 7].isfinite().any()
    got[1, 3:, 7] = want[1, 3:, 7]
    assert torch.equal(got, want)


@pytest.mark.parametrize("ps,top,dt,Hq,Hkv,D", [(16, 5, torch.float16, 10, 2, 64), (32, 3, torch.bfloat16, 25, 5, 64),
                                                (64, 4, torch.float16, 8, 1, 128), (128, 2, torch.float16, 12, 1, 64)])
def test_attention_listed_pages(ps, top, dt, Hq, Hkv, D):
    lens = [0, 1, ps, ps + 1, 7 * ps - 5, 9 * ps, 20 * ps + 3]
    k, v, table = R.make_pool(lens, ps, Hkv, D, dt, seed=8)
    g = torch.Generator().manual_seed(9)
    q = torch.randn(len(lens), Hq, D, generator=g).to(dt)
    idx = torch.full((len(lens), Hkv, top), -1, dtype=torch.int32)
    for b, n in enumerate(lens):
        total = -(-n // ps)
        for h in range(Hkv):
            pick = torch.randperm(max(total, 1), generator=g)[:min(top, total)]
            idx[b, h, :len(pick)] = pick.to(torch.int32)      # in no order
    idx[5, 0, 0] = -1                                          # a hole
    idx[6, Hkv - 1, top - 1] = 10 ** 6                         # no page of the sequence
    idx[4, 0, 1] = idx[4, 0, 0]                                # listed twice
    ref = R.attention(k, v, table, lens, q, 0.3, page_idx=idx)
    got, lse, status = run_attention(k, v, table, lens, q, page_idx=idx, scale=0.3)
    assert status == H.OK
    check_attention(got, lse, ref, v, top * ps, dt, torch.float32, D)


@pytest.mark.parametrize("Hq,Hkv,D,ps,dt,lens", [
    (25, 5, 64, 64, torch.float16, [20011]),                      # one sequence over every CTA
    (4, 1, 128, 16, torch.bfloat16, [9000, 3, 12345, 700]),
    (16, 1, 64, 32, torch.float16, [30000]),
    (10, 2, 64, 16, torch.float16, [(i * 37) % 150 for i in range(700)]),   # many short ones, several a thread
])
def test_attention_split_and_joined(Hq, Hkv, D, ps, dt, lens):
    k, v, table = R.make_pool(lens, ps, Hkv, D, dt, seed=10)
    q = (torch.randn(len(lens), Hq, D, generator=torch.Generator().manual_seed(11)) * 2).to(dt)
    ref = R.attention(k, v, table, lens, q, D ** -0.5)
    got, lse, status = run_attention(k, v, table, lens, q)
    assert status == H.OK
    check_attention(got, lse, ref, v, max(lens), dt, torch.float32, D)
    again, lse2, _ = run_attention(k, v, table, lens, q)
    assert torch.equal(got, again) and torch.equal(lse, lse2)      # bit for bit


@pytest.mark.parametrize("D,Hq,Hkv,dt", [(64, 25, 5, torch.float16), (128, 16, 4, torch.bfloat16),
                                         (64, 12, 1, torch.float16)])
def test_attention_items_cut_between_groups_and_ctas(D, Hq, Hkv, dt):
    """About two items per CTA: nearly every CTA ends one, begins one and cuts others between its
    groups, all at once.  Lengths shift from round to round, and every round must repeat itself."""
    for r in range(6):
        lens = [(977 * (i + 1) * (r + 1)) % 1800 for i in range(64)]
        k, v, table = R.make_pool(lens, 64, Hkv, D, dt, seed=80 + r)
        q = torch.randn(64, Hq, D, generator=torch.Generator().manual_seed(81 + r)).to(dt)
        ref = R.attention(k, v, table, lens, q, D ** -0.5)
        first = None
        for _ in range(4):
            got, lse, status = run_attention(k, v, table, lens, q)
            assert status == H.OK
            check_attention(got, lse, ref, v, max(lens), dt, torch.float32, D)
            assert first is None or torch.equal(first, got)
            first = got


def test_attention_growing_maximum():
    """Scores that rise along the sequence, so every tile rescales what came before."""
    n, dt, D = 5000, torch.float16, 64
    k, v, table = R.make_pool([n], 64, 1, D, dt, seed=12)
    q = torch.zeros(1, 3, D, dtype=dt)
    q[0, :, 0] = torch.tensor([8.0, -8.0, 1.0])
    for p in range(n):
        k[table[0, p // 64].long(), 0, p % 64, 0] = p / 100.0
    ref = R.attention(k, v, table, [n], q, 0.125)
    got, lse, status = run_attention(k, v, table, [n], q)
    assert status == H.OK
    check_attention(got, lse, ref, v, n, dt, torch.float32, D)


@pytest.mark.parametrize("D,Hq,Hkv,dt", [(64, 5, 1, torch.float16), (128, 9, 1, torch.float16), (64, 2, 2, torch.bfloat16)])
def test_attention_small_probabilities_add_up(D, Hq, Hkv, dt):
    """One key of every 16 takes nearly all of the weight and has the value 0; the others, each
    e^-17.5 of it (below half of fp16's smallest step), make the whole result.  Values are not
    negative, so the bound of check_attention holds relative to the result itself: it is
    c sum_j p_j |v_j| before max|v| is put in its place."""
    n, ps = 1500, 64
    k, v, table = R.make_pool([n], ps, Hkv, D, dt, seed=31)
    k[k.isfinite()] = 0
    v[v.isfinite()] = v[v.isfinite()].abs().clamp(0.25, 2)
    big = torch.arange(0, n, 16)
    page = table[0].long()[big // ps]
    k[page, :, big % ps, 0] = 1
    v[page, :, big % ps] = 0
    q = torch.zeros(1, Hq, D, dtype=dt)
    q[..., 0] = 17.5
    out, _, size = R.attention(k, v, table, [n], q, 1.0)
    got, _, status = run_attention(k, v, table, [n], q, scale=1.0)
    assert status == H.OK
    small = 2.0 ** -40 * math.exp(17.5) if dt == torch.float16 else 0   # of the parts of p
    c = 2 * (2 * D + 8) * U * size[..., None] + (2 * (n + 64) + 8) * U + half_step(dt) ** 2 + U + small
    err = (got.double() - out).abs()
    assert (err <= (c + U) * out).all(), f"worst {float((err / out).max()):.2e} of the result"


def test_attention_pool_halves_and_sliced_table():
    """K and V as halves of one tensor's pages, a table that is a slice of a wider one, lengths
    that are a slice of a longer vector, and a batch of nothing but empty sequences."""
    ps, Hq, Hkv, D, dt, lens = 32, 10, 2, 64, torch.bfloat16, [100, 3, 260]
    k, v, table = R.make_pool(lens, ps, Hkv, D, dt, seed=15)
    both = torch.stack([k, v], 1).cuda()                       # [n_pages, 2, Hkv, page_size, D]
    cache = H.PagedCache(both[:, 0], both[:, 1])
    wide = torch.full((3, table.shape[1] + 5), -9, dtype=torch.int32)
    wide[:, 2:2 + table.shape[1]] = table
    tb = wide.cuda()[:, 2:2 + table.shape[1]]
    ln = torch.tensor([7, 7] + lens + [7], dtype=torch.int32, device="cuda")[2:5]
    q = torch.randn(3, Hq, D, generator=torch.Generator().manual_seed(16)).to(dt)
    ws = workspace(cache, 3, Hq, table.shape[1])
    out, lse = torch.empty(3, Hq, D, device="cuda"), torch.empty(3, Hq, device="cuda")
    H.paged_attention(cache, q.cuda(), tb, ln, out, ws, lse=lse)
    assert H.status_read(ws) == H.OK
    check_attention(out.cpu(), lse.cpu(), R.attention(k, v, table, lens, q, D ** -0.5), v, 260, dt, torch.float32, D)
    H.paged_attention(cache, q.cuda(), tb, torch.zeros_like(ln), out, ws, lse=lse)
    assert H.status_read(ws) == H.OK and (out == 0).all() and (lse == -math.inf).all()
    kv = torch.randn(3, Hkv, D, device="cuda").to(dt)          # append through the same views
    H.paged_append(cache, tb, ln - 1, kv, kv, ws, rope_base=0.0)
    assert H.status_read(ws) == H.OK
    for b, n in enumerate(lens):
        page, row = int(table[b, (n - 1) // ps]), (n - 1) % ps
        assert torch.equal(both[page, 0, :, row], kv[b]) and torch.equal(both[page, 1, :, row], kv[b])


def test_attention_strided_rows_and_bad_lengths():
    """Queries and outputs inside wider rows; lengths and pages that do not exist are recorded
    and change nothing else."""
    lens, ps, Hq, Hkv, D, dt = [70, 50, 33], 16, 4, 2, 64, torch.float16
    k, v, table = R.make_pool(lens, ps, Hkv, D, dt, seed=13)
    g = torch.Generator().manual_seed(14)
    wide = torch.randn(3, Hq * D + 72, generator=g).to(dt).cuda()
    q = wide[:, 8:8 + Hq * D].view(3, Hq, D)
    cache = H.PagedCache(k.cuda(), v.cuda())
    ws = workspace(cache, 3, Hq, table.shape[1])
    buf = torch.full((3, Hq * D + 40), 7.0, device="cuda")
    out = buf[:, 16:16 + Hq * D].view(3, Hq, D)
    tb = table.cuda()
    H.paged_attention(cache, q, tb, torch.tensor(lens, dtype=torch.int32, device="cuda"), out, ws)
    assert H.status_read(ws) == H.OK
    ref = R.attention(k, v, table, lens, q.cpu(), 0.125)
    check_attention(out.cpu(), None, ref, v, 70, dt, torch.float32, D)
    assert (buf[:, :16] == 7).all() and (buf[:, 16 + Hq * D:] == 7).all()
    # too long: clamped to the table (5 pages); negative: empty
    H.paged_attention(cache, q[1:2], tb[1:2], torch.tensor([-3], dtype=torch.int32, device="cuda"),
                      out[1:2], ws)
    assert H.status_read(ws) == H.ERR_INVALID_ARG and (out[1] == 0).all()
    H.paged_attention(cache, q[:1], tb[:1], torch.tensor([81], dtype=torch.int32, device="cuda"), out[:1], ws)
    assert H.status_read(ws) == H.ERR_INVALID_ARG
    # a page outside the pool: its positions are skipped
    for bad in (-1, cache.c.n_pages, 2 ** 31 - 1):
        t2 = table.clone()
        t2[0, 2] = bad
        H.paged_attention(cache, q, t2.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), out, ws)
        assert H.status_read(ws) == H.ERR_INVALID_ARG
        idx = torch.tensor([0, 1, 3, 4, -1], dtype=torch.int32).expand(3, Hkv, 5)
        ref2 = R.attention(k, v, table, [70, 0, 0], q.cpu(), 0.125, page_idx=idx)
        check_attention(out[:1].cpu(), None, tuple(t[:1] for t in ref2), v, 70, dt, torch.float32, D)
        check_attention(out[1:].cpu(), None, tuple(t[1:] for t in ref), v, 70, dt, torch.float32, D)


# ---------------------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------------------
def run_append(ps, Hq, Hkv, D, dt, src, start, new, base, bounds=True, with_q=True, layout="page_head_row", seed=20,
               tail=2):
    """Append `new` tokens per sequence behind `start`; returns everything before and after."""
    lens = [s + n for s, n in zip(start, new)]
    k, v, table = R.make_pool(lens, ps, Hkv, D, dt, seed=seed, layout=layout, poison=False)
    g = torch.Generator().manual_seed(seed + 1)
    T = sum(new) + tail                       # rows behind the last sequence
    P = (Hq + 2 * Hkv) * D
    proj = (torch.randn(T, P + 64, generator=g) * 1.5).to(src)
    lo, hi = (k.amin(2), k.amax(2)) if bounds else (None, None)
    dev = lambda t: None if t is None else R.to_gpu(t)
    cache = H.PagedCache(dev(k), dev(v), dev(lo), dev(hi))
    pg = proj.cuda()
    cols = lambda t, a, h: t[:, a * D:(a + h) * D].view(T, h, D)
    q_out = torch.full((T, Hq, D), 5.0, dtype=dt, device="cuda") if with_q else None
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    ws = H.alloc_workspace(256)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    H.paged_append(cache, table.cuda(), i32(start), cols(pg, Hq, Hkv), cols(pg, Hq + Hkv, Hkv), ws,
                   q=cols(pg, 0, Hq) if with_q else None, q_out=q_out, cu_new=i32(cu), rope_base=base)
    torch.cuda.synchronize()
    return dict(k0=k, v0=v, lo0=lo, hi0=hi, table=table, proj=proj, cache=cache, q_out=q_out, cu=cu,
                status=H.status_read(ws), q=cols(proj, 0, Hq), k=cols(proj, Hq, Hkv), v=cols(proj, Hq + Hkv, Hkv))


def check_append(r, ps, dt, start, new, base):
    kw, vw = r["k0"].double(), r["v0"].double().clone()
    slack = torch.zeros_like(kw)
    kw = kw.clone()
    vw = r["v0"].clone()
    k_got, v_got = r["cache"].t["k"].cpu(), r["cache"].t["v"].cpu()
    u16, sub = half_step(dt), (2.0 ** -25 if dt == torch.float16 else 0.0)
    for b, (s, n) in enumerate(zip(start, new)):
        if n == 0:
            continue
        rows = slice(r["cu"][b], r["cu"][b + 1])
        pos = list(range(s, s + n))
        kr = R.rotate(r["k"][rows], pos, base)
        mag = r["k"][rows].double().abs()
        mag = mag + torch.roll(mag, mag.shape[-1] // 2, -1)
        p = torch.tensor(pos)
        page = r["table"][b].long()[p // ps]
        kw[page, :, p % ps] = kr
        slack[page, :, p % ps] = 8 * U * mag + u16 * kr.abs() + sub
        vw[page, :, p % ps] = r["v"][rows].to(dt)
        if r["q_out"] is not None:
            qr = R.rotate(r["q"][rows], pos, base)
            qm = r["q"][rows].double().abs()
            qm = qm + torch.roll(qm, qm.shape[-1] // 2, -1)
            assert ((r["q_out"][rows].cpu().double() - qr).abs() <= 8 * U * qm + u16 * qr.abs() + sub).all()
    assert torch.equal(v_got, vw)
    assert ((k_got.double() - kw).abs() <= slack).all()      # 0 where nothing was appended
    if r["q_out"] is not None:
        assert (r["q_out"][r["cu"][-1]:] == 5).all()         # rows behind the last sequence
    if r["lo0"] is not None:
        lo, hi = r["lo0"].clone(), r["hi0"].clone()
        for b, (s, n) in enumerate(zip(start, new)):
            for j in range(s // ps, -(-(s + n) // ps) if n else 0):
                pg = int(r["table"][b, j])
                a, e = max(s, j * ps) - j * ps, min(s + n, (j + 1) * ps) - j * ps
                rows = k_got[pg, :, a:e]
                l, h = rows.amin(1), rows.amax(1)
                lo[pg] = torch.minimum(lo[pg], l) if a > 0 else l
                hi[pg] = torch.maximum(hi[pg], h) if a > 0 else h
        assert torch.equal(r["cache"].t["k_lo"].cpu(), lo) and torch.equal(r["cache"].t["k_hi"].cpu(), hi)


@pytest.mark.parametrize("Hq,Hkv,D,ps,dt,src,base,layout", [
    (25, 5, 64, 64, torch.float16, torch.float32, 10000.0, "page_head_row"),
    (25, 5, 64, 16, torch.bfloat16, torch.bfloat16, 10000.0, "page_row_head"),
    (4, 2, 64, 32, torch.float16, torch.float16, 0.0, "page_head_row"),
    (32, 8, 128, 16, torch.bfloat16, torch.float32, 500000.0, "head_page_row"),
    (9, 1, 128, 128, torch.float16, torch.bfloat16, 10000.0, "page_head_row"),
    (6, 6, 128, 256, torch.bfloat16, torch.float16, 1e6, "page_row_head"),
])
def test_append(Hq, Hkv, D, ps, dt, src, base, layout):
    start = [0, 5, ps - 1, ps, 3 * ps + 7, 0, 17, 1000]
    new = [1, 0, 2, ps, 2 * ps + 3, 3 * ps, 1, 1]
    for bounds in (True, False):
        r = run_append(ps, Hq, Hkv, D, dt, src, start, new, base, bounds, with_q=bounds, layout=layout)
        assert r["status"] == H.OK
        check_append(r, ps, dt, start, new, base)


@pytest.mark.parametrize("Hq,Hkv,D,ps,dt,src", [(4, 2, 64, 16, torch.float16, torch.float32),
                                                (16, 1, 128, 32, torch.bfloat16, torch.float32)])
def test_append_many_short_sequences(Hq, Hkv, D, ps, dt, src):
    """More sequences than a warp looks through at once, runs of them without new tokens, more
    items than CTAs; the widest group's rows need the largest stage."""
    start = [(i * 13) % 70 for i in range(500)]
    new = [0 if i % 7 in (1, 2) or 100 <= i < 170 else (i * 5) % 40 for i in range(500)]
    r = run_append(ps, Hq, Hkv, D, dt, src, start, new, 10000.0)
    assert r["status"] == H.OK
    check_append(r, ps, dt, start, new, 10000.0)


def test_append_one_token_each_and_far_positions():
    """Without cu_new; positions where an fp32 angle would have lost its phase."""
    ps, Hkv, D, dt = 64, 2, 64, torch.float16
    start = [0, 63, 64, 1_000_003]
    pool = torch.zeros(6, Hkv, ps, D, dtype=dt, device="cuda")
    cache = H.PagedCache(pool, pool.clone())
    width = 1_000_003 // ps + 1
    table = torch.full((4, width), -1, dtype=torch.int32)
    for b, s in enumerate(start):
        table[b, s // ps] = b
    g = torch.Generator().manual_seed(30)
    k, v = torch.randn(4, Hkv, D, generator=g), torch.randn(4, Hkv, D, generator=g)
    ws = H.alloc_workspace(256)
    H.paged_append(cache, table.cuda(), torch.tensor(start, dtype=torch.int32, device="cuda"), k.cuda(), v.cuda(), ws)
    assert H.status_read(ws) == H.OK
    for b, s in enumerate(start):
        ref = R.rotate(k[b:b + 1], [s], 10000.0)[0]
        mag = k[b].double().abs()
        mag = mag + torch.roll(mag, D // 2, -1)
        got = cache.t["k"][b, :, s % ps].cpu().double()
        assert ((got - ref).abs() <= 8 * U * mag + half_step(dt) * ref.abs() + 2.0 ** -25).all()
        assert torch.equal(cache.t["v"][b, :, s % ps].cpu(), v[b].to(dt))


def test_append_in_place_and_of_nothing():
    """Queries rotated where they are, in both kernels; a call without tokens changes nothing."""
    ps, Hq, Hkv, D, dt = 16, 8, 2, 64, torch.float16
    cache = H.PagedCache.zeros(20, ps, Hkv, D, dt, bounds=True)
    table = torch.arange(20, dtype=torch.int32, device="cuda").view(2, 10)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ws = H.alloc_workspace(256)
    for new in ((1, 1), (70, 33)):
        T = sum(new)
        q, k = torch.randn(T, Hq, D, device="cuda").to(dt), torch.randn(T, Hkv, D, device="cuda").to(dt)
        want = torch.empty_like(q)
        cu = None if T == 2 else i32(0, new[0], T)
        H.paged_append(cache, table, i32(3, 40), k, k, ws, q=q, q_out=want, cu_new=cu)
        H.paged_append(cache, table, i32(3, 40), k, k, ws, q=q, q_out=q, cu_new=cu)
        assert torch.equal(q, want)
    before = cache.t["k"].clone()
    H.paged_append(cache, table, i32(0, 0), k[:0], k[:0], ws, q=q[:0], q_out=q[:0], cu_new=i32(0, 0, 0))
    H.paged_append(cache, table, i32(0, 0), k, k, ws, q=q, q_out=want, cu_new=i32(0, 0, 0))
    assert torch.equal(before, cache.t["k"]) and H.status_read(ws) == H.OK


def test_append_skips_what_has_no_place():
    """A position beyond the table, a bad page, a negative start: recorded, nothing stored for
    them, the others as ever.  Out-of-range fp16 values are recorded."""
    ps, Hkv, D, dt = 16, 1, 64, torch.float16
    pool = torch.zeros(4, Hkv, ps, D, dtype=dt, device="cuda")
    cache = H.PagedCache(pool, pool.clone())
    table = torch.tensor([[0, 9], [1, -1], [2, 3], [3, 2]], dtype=torch.int32, device="cuda")
    k = torch.ones(4, Hkv, D, device="cuda")
    ws = H.alloc_workspace(256)
    q_out = torch.zeros(4, 1, D, dtype=dt, device="cuda")
    start = torch.tensor([16, 32, -1, 3], dtype=torch.int32, device="cuda")
    H.paged_append(cache, table, start, k, k, ws, q=k, q_out=q_out)
    assert H.status_read(ws) == H.ERR_INVALID_ARG
    want = torch.zeros_like(pool)
    want[3, 0, 3] = 1
    assert torch.equal(cache.t["v"], want)
    assert (q_out[2] == 0).all() and (q_out[[0, 1, 3]] != 0).any(-1).all()
    # cu_new that points outside the rows
    for cu in ([0, 1, 2, 3, 9], [0, 2, 1, 3, 4], [-1, 1, 2, 3, 4]):
        H.paged_append(cache, table, torch.full((4,), 5, dtype=torch.int32, device="cuda"), k, k, ws,
                       cu_new=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert H.status_read(ws) == H.ERR_INVALID_ARG
    H.paged_append(cache, table, torch.zeros(4, dtype=torch.int32, device="cuda"), k * 7e4, k, ws)
    assert H.status_read(ws) == H.ERR_FP16_RANGE


# ---------------------------------------------------------------------------------------
# select
# ---------------------------------------------------------------------------------------
def run_select(lo, hi, table, lens, q, ps, top, n_first, n_last):
    n_pages, Hkv, D = lo.shape
    k = torch.zeros(n_pages, Hkv, ps, D, dtype=lo.dtype, device="cuda")
    cache = H.PagedCache(k, k, lo.cuda(), hi.cuda())
    B, Hq = q.shape[:2]
    ws = workspace(cache, B, Hq, table.shape[1])
    idx = torch.full((B, Hkv, top), 77, dtype=torch.int32, device="cuda")
    H.paged_select(cache, q.cuda(), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), idx, ws,
                   n_first=n_first, n_last=n_last)
    return idx.cpu(), H.status_read(ws)


@pytest.mark.parametrize("Hq,Hkv,D,ps,dt", [(25, 5, 64, 64, torch.float16), (4, 2, 64, 16, torch.bfloat16),
                                            (32, 4, 128, 32, torch.bfloat16), (16, 1, 128, 16, torch.float16)])
@pytest.mark.parametrize("top,nf,nl", [(1, 0, 1), (5, 2, 1), (3, 2, 1), (40, 0, 0), (70, 3, 2)])
def test_select(Hq, Hkv, D, ps, dt, top, nf, nl):
    pages = [0, 1, 3, 5, 6, 64, 65, 100, 600]
    lens = [n * ps - (3 if i % 2 and n else 0) for i, n in enumerate(pages)]
    g = torch.Generator().manual_seed(40)
    n_pages = sum(pages) + 2
    mid = torch.randn(n_pages, Hkv, D, generator=g)
    wid = torch.rand(n_pages, Hkv, D, generator=g)
    lo, hi = (mid - wid).to(dt), (mid + wid).to(dt)
    perm = torch.randperm(n_pages, generator=g).to(torch.int32)
    table = torch.full((len(pages), max(pages)), -1, dtype=torch.int32)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = perm[at:at + n]
        at += n
    q = torch.randn(len(pages), Hq, D, generator=g).to(dt)
    got, status = run_select(lo, hi, table, lens, q, ps, top, nf, nl)
    assert status == H.OK
    for b, n in enumerate(pages):
        sc = R.scores(lo, hi, table[b, :n], q[b])
        for h in range(Hkv):
            assert got[b, h].tolist() == R.select(sc[h].tolist(), nf, nl, top), (b, h)


@pytest.mark.parametrize("n,kinds", [(50, 1), (50, 2), (3000, 3), (3000, 1), (16384, 40)])
def test_select_ties_go_to_the_lowest_page(n, kinds):
    """Few distinct pages, values exact in 64 bits: ranks rest on ties; scores of both signs,
    subnormal values and -0 among them."""
    dt, D = torch.float16, 64
    g = torch.Generator().manual_seed(41)
    lo = torch.randint(-3, 3, (kinds, 1, D), generator=g).to(dt)
    hi = lo + torch.randint(0, 3, (kinds, 1, D), generator=g).to(dt)
    lo[0], hi[0] = -0.0, 2.0 ** -24
    table = torch.randint(0, kinds, (1, n), generator=g).to(torch.int32)
    q = torch.randint(-2, 3, (1, 3, D), generator=g).to(dt)
    for top, nf, nl in ((1, 0, 0), (17, 3, 4), (49, 0, 1), (min(n - 1, 2000), 1, 1)):
        got, status = run_select(lo, hi, table, [n * 16 - 1], q, 16, top, nf, nl)
        assert status == H.OK
        sc = R.scores(lo, hi, table[0], q[0])[0].tolist()
        assert got[0, 0].tolist() == R.select(sc, nf, nl, top)


def test_select_records_bad_lengths_and_pages():
    dt, D = torch.float16, 64
    lo = torch.zeros(4, 1, D, dtype=dt)
    hi = torch.ones(4, 1, D, dtype=dt)
    q = torch.ones(1, 1, D, dtype=dt)
    table = torch.tensor([[0, 99, 2, 1]], dtype=torch.int32)
    got, status = run_select(lo, hi, table, [64], q, 16, 2, 0, 0)
    assert status == H.ERR_INVALID_ARG and got[0, 0].tolist() == [0, 2]
    got, status = run_select(lo, hi, table[:, :1], [64], q, 16, 2, 0, 0)
    assert status == H.ERR_INVALID_ARG and got[0, 0].tolist() == [0, -1]
    got, status = run_select(lo, hi, table[:, :1], [-5], q, 16, 2, 0, 0)
    assert status == H.ERR_INVALID_ARG and got[0, 0].tolist() == [-1, -1]


# ---------------------------------------------------------------------------------------
# together, and how calls are made
# ---------------------------------------------------------------------------------------
def test_a_run_of_appends_selections_and_attention():
    """Prompts of different lengths, then decode steps: each appends a token, chooses pages and
    attends over them and over everything.  The pool's own keys are the reference's input."""
    Hq, Hkv, D, ps, dt, top = 10, 2, 64, 16, torch.float16, 6
    prompts, steps = [130, 1, 47, 300], 5
    B = len(prompts)
    width = (max(prompts) + steps) // ps + 1
    n_pages = B * width
    cache = H.PagedCache.zeros(n_pages, ps, Hkv, D, dt, bounds=True)
    g = torch.Generator().manual_seed(50)
    table = torch.randperm(n_pages, generator=g).to(torch.int32).view(B, width).cuda()
    ws = workspace(cache, B, Hq, width)
    T = sum(prompts)
    rnd = lambda n, h: torch.randn(n, h, D, generator=g).to(torch.bfloat16).cuda()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0] + [sum(prompts[:i + 1]) for i in range(B)], dtype=torch.int32, device="cuda")
    H.paged_append(cache, table, lens, rnd(T, Hkv), rnd(T, Hkv), ws, cu_new=cu)
    lens += torch.tensor(prompts, dtype=torch.int32, device="cuda")
    q = torch.empty(B, Hq, D, dtype=dt, device="cuda")
    idx = torch.empty(B, Hkv, top, dtype=torch.int32, device="cuda")
    out = [torch.empty(B, Hq, D, device="cuda") for _ in range(2)]
    lse = torch.empty(B, Hq, device="cuda")
    for _ in range(steps):
        H.paged_append(cache, table, lens, rnd(B, Hkv), rnd(B, Hkv), ws, q=rnd(B, Hq), q_out=q)
        lens += 1
        H.paged_select(cache, q, table, lens, idx, ws, n_first=1, n_last=2)
        H.paged_attention(cache, q, table, lens, out[0], ws, page_idx=idx)
        H.paged_attention(cache, q, table, lens, out[1], ws, lse=lse)
        assert H.status_read(ws) == H.OK
        kc, vc, tc, qc, ic = (t.cpu() for t in (cache.t["k"], cache.t["v"], table, q, idx))
        n = lens.tolist()
        for b in range(B):
            pages = -(-n[b] // ps)
            for j in range(pages):
                rows = kc[tc[b, j].long(), :, :min(ps, n[b] - j * ps)]
                assert torch.equal(cache.t["k_lo"][tc[b, j].long()].cpu(), rows.amin(1))
                assert torch.equal(cache.t["k_hi"][tc[b, j].long()].cpu(), rows.amax(1))
            sc = R.scores(cache.t["k_lo"].cpu(), cache.t["k_hi"].cpu(), tc[b, :pages], qc[b])
            for h in range(Hkv):
                assert ic[b, h].tolist() == R.select(sc[h].tolist(), 1, 2, top)
        ref = R.attention(kc, vc, tc, n, qc, D ** -0.5, page_idx=ic)
        check_attention(out[0].cpu(), None, ref, vc, top * ps, dt, torch.float32, D)
        ref = R.attention(kc, vc, tc, n, qc, D ** -0.5)
        check_attention(out[1].cpu(), lse.cpu(), ref, vc, max(n), dt, torch.float32, D)


def test_captured_step_serves_later_lengths_and_graphs_share_a_workspace():
    """One captured step (append, select, attend) replayed as the sequences grow, in turn with
    a second graph on the same workspace, equals the eager calls bit for bit."""
    Hq, Hkv, D, ps, dt, top, B = 25, 5, 64, 32, torch.float16, 4, 3
    width = 40
    g = torch.Generator().manual_seed(60)
    table = torch.randperm(B * width, generator=g).to(torch.int32).view(B, width).cuda()
    k0 = torch.randn(B * width, Hkv, ps, D, generator=g).to(dt)
    v0 = torch.randn(B * width, Hkv, ps, D, generator=g).to(dt)
    start0 = torch.tensor([95, 0, 1100], dtype=torch.int32)
    feed = [torch.randn(B, (Hq + 2 * Hkv) * D, generator=g).cuda() for _ in range(4)]

    class Step:
        def __init__(self, ws=None):
            self.cache = H.PagedCache(k0.cuda(), v0.cuda(), k0.amin(2).cuda(), k0.amax(2).cuda())
            self.ws = workspace(self.cache, B, Hq, width) if ws is None else ws
            self.lens = start0.cuda()
            self.x = torch.zeros(B, (Hq + 2 * Hkv) * D, device="cuda")
            self.q = torch.zeros(B, Hq, D, dtype=dt, device="cuda")
            self.idx = torch.zeros(B, Hkv, top, dtype=torch.int32, device="cuda")
            self.out = torch.zeros(2, B, Hq, D, device="cuda")

        def __call__(self):
            c = lambda a, h: self.x[:, a * D:(a + h) * D].view(B, h, D)
            H.paged_append(self.cache, table, self.lens, c(Hq, Hkv), c(Hq + Hkv, Hkv), self.ws, q=c(0, Hq),
                           q_out=self.q)
            self.lens += 1
            H.paged_select(self.cache, self.q, table, self.lens, self.idx, self.ws)
            H.paged_attention(self.cache, self.q, table, self.lens, self.out[0], self.ws, page_idx=self.idx)
            H.paged_attention(self.cache, self.q, table, self.lens, self.out[1], self.ws, n_meta=8, window=100)

    eager, a = Step(), Step()
    b = Step(a.ws)
    graphs = []
    for s in (a, b):
        gr = torch.cuda.CUDAGraph()
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st), torch.cuda.graph(gr, stream=st):
            s()
        graphs.append(gr)
    torch.cuda.synchronize()
    for x in feed:
        for s in (eager, a, b):
            s.x.copy_(x)
        eager()
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for s in (a, b):
            assert torch.equal(s.out, eager.out) and torch.equal(s.idx, eager.idx)
            assert torch.equal(s.cache.t["k"], eager.cache.t["k"]) and torch.equal(s.cache.t["k_lo"], eager.cache.t["k_lo"])
    assert H.status_read(a.ws) == H.OK and H.status_read(eager.ws) == H.OK


def test_two_streams_with_a_workspace_each():
    lens, ps, Hq, Hkv, D, dt = [3000, 10, 777], 64, 25, 5, 64, torch.float16
    k, v, table = R.make_pool(lens, ps, Hkv, D, dt, seed=70)
    cache = H.PagedCache(k.cuda(), v.cuda())
    q = torch.randn(2, 3, Hq, D, generator=torch.Generator().manual_seed(71)).to(dt).cuda()
    tb, ln = table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    want = [torch.zeros(3, Hq, D, device="cuda") for _ in range(2)]
    got = [torch.zeros(3, Hq, D, device="cuda") for _ in range(2)]
    wss = [workspace(cache, 3, Hq, table.shape[1]) for _ in range(2)]
    for i in range(2):
        H.paged_attention(cache, q[i], tb, ln, want[i], wss[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(20):
        for i, s in enumerate(streams):
            H.paged_attention(cache, q[i], tb, ln, got[i], wss[i], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    assert all(H.status_read(w) == H.OK for w in wss)


def test_binding_refuses_what_it_can_see():
    cache = H.PagedCache.zeros(4, 16, 2, 64)
    ws = workspace(cache, 1, 4, 2)
    tb = torch.zeros(1, 2, dtype=torch.int32, device="cuda")
    ln = torch.ones(1, dtype=torch.int32, device="cuda")
    q = torch.zeros(1, 4, 64, dtype=torch.float16, device="cuda")
    out = torch.zeros(1, 4, 64, device="cuda")
    good = dict(cache=cache, q=q, table=tb, seq_lens=ln, out=out, ws=ws)
    H.paged_attention(**good)
    for bad in (dict(q=q.float()), dict(q=q.cpu()), dict(table=tb.long()), dict(seq_lens=ln.long()),
                dict(seq_lens=ln.expand(2)), dict(out=out[:, :2]), dict(ws=ws[:512]), dict(lse=out[..., 0].half()),
                dict(page_idx=torch.zeros(1, 2, 3, device="cuda")), dict(n_meta=4), dict(window=-1),
                dict(scale=math.nan), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2)),
                dict(out=out.double()), dict(q=q[:, :3], out=out[:, :3]), dict(out=q)):
        with pytest.raises(H.HymbaError):
            H.paged_attention(**{**good, **bad})
    with pytest.raises(H.HymbaError):                     # no page bounds
        H.paged_select(cache, q, tb, ln, torch.zeros(1, 2, 1, dtype=torch.int32, device="cuda"), ws)
    kv = torch.zeros(1, 2, 64, device="cuda")
    for bad in (dict(v=None), dict(q=q), dict(k=kv[:, :1]), dict(k=kv.half()), dict(rope_base=-1.0),
                dict(cu_new=ln), dict(start=ln.float())):
        with pytest.raises(H.HymbaError):
            H.paged_append(**{**dict(cache=cache, table=tb, start=ln, k=kv, v=kv, ws=ws), **bad})
    with pytest.raises(H.HymbaError):
        H.PagedCache(cache.t["k"], cache.t["v"].transpose(0, 1))
    assert H.status_read(ws) == H.OK
