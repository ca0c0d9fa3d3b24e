"""The paged attention where the bounds of test_gpu_paged are too wide to see a mistake: sums that
are exact, so that one lost, doubled or misplaced position shows at any length; bounds from the
kernel's own order of sums; the third part of a bf16 pool's probabilities."""
import math

import pytest
import torch

from hybrid_attention_ssm_b200 import hymba as H
from tests import paged_ref as R
from tests.test_gpu_paged import U, half_step, run_attention

pytestmark = pytest.mark.gpu
SPLIT = [  # Hq, Hkv, D, page, dtype, lengths: one sequence over every CTA, several, many short ones
    (25, 5, 64, 64, torch.float16, [20011]),
    (8, 1, 64, 16, torch.bfloat16, [131073]),
    (16, 1, 64, 32, torch.float16, [30000]),
    (9, 1, 128, 64, torch.bfloat16, [40000, 64, 1]),
    (4, 1, 128, 16, torch.bfloat16, [9000, 3, 12345, 700]),
    (10, 2, 64, 128, torch.float16, [(i * 37) % 150 for i in range(700)]),
    (25, 5, 64, 64, torch.float16, [(977 * (i + 1)) % 1800 for i in range(64)]),
]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.lib()


@pytest.mark.parametrize("Hq,Hkv,D,ps,dt,lens", SPLIT)
@pytest.mark.parametrize("M,W", [(0, 0), (70, 1000)])
def test_equal_scores_sum_exactly(Hq, Hkv, D, ps, dt, lens, M, W):
    """Queries of zero: every weight is 1, and with small whole numbers as values every partial
    sum is one too, below 2^24: nothing is rounded before the division (1 / l and the product,
    half a step of 2^-24 each).  Tile t's positions have their values in channel t % D alone, so
    a tile that is lost, doubled or read from another place changes a channel by far more than
    that, whatever the length; the number of positions shows in the lse."""
    k, v, table = R.make_pool(lens, ps, Hkv, D, dt, seed=110)
    zero = v.isfinite()
    v[zero] = 0
    want = torch.zeros(len(lens), Hkv, D, dtype=torch.float64)
    count = torch.zeros(len(lens), dtype=torch.float64)
    for b, n in enumerate(lens):
        pos = torch.arange(n)
        page, tile = table[b].long()[pos // ps], pos // 64
        val = 1 + (pos * 7 + tile * 3) % 13
        for h in range(Hkv):
            v[page, h, pos % ps, (tile + h) % D] = val.to(dt)
        seen = (pos < M) | (pos >= n - W) if W else pos >= 0
        count[b] = seen.sum()
        for h in range(Hkv):
            want[b, h].index_add_(0, (tile + h)[seen] % D, val[seen].double())
    assert want.max() < 2 ** 24
    want = want / count.clamp(min=1)[:, None, None]
    q = torch.zeros(len(lens), Hq, D, dtype=dt)
    got, lse, status = run_attention(k, v, table, lens, q, n_meta=M, window=W)
    assert status == H.OK
    want = want.repeat_interleave(Hq // Hkv, 1)
    assert ((got.double() - want).abs() <= (2 * U + U * U) * want).all()
    ref = count.log()[:, None].expand(-1, Hq)        # ln 2 * log2 n: log2f 1 ulp, the constant and the product
    none = count == 0
    assert (lse[none] == -math.inf).all()
    assert ((lse.double() - ref).abs()[~none] <= 5 * U * ref[~none] + 1e-30).all()


@pytest.mark.parametrize("Hq,Hkv,D,ps,dt,lens", SPLIT)
def test_split_sums_within_the_bound_of_their_order(Hq, Hkv, D, ps, dt, lens):
    """Random scores, with the length of the real chain of sums in the place of n: a group adds its
    tiles one by one (per tile a rescaling, and a matrix instruction's sum of 16 products for
    each part of p: at most 4 steps of 2 u), then come the merges of 4 warps, of a CTA's 2 to 6 group
    parts and of at most `parts` CTAs (3 steps of u each), where a share is the call's tiles over 148
    CTAs.  Relative to sum_j p_j |v_j| of the row itself:
      c = 2 d + 2 (4 tiles + 3 (10 + parts)) u + 8 u + u16^2 (u16^3: bf16 pool, fp32 output)
    with d the error of the scores as in test_gpu_paged, and in fp16 2^-40 of the largest p on top
    for each key (its parts are of 2^15 p).  A tile that is left out exceeds this at every length
    here: checked on the reference, in the places where it matters least."""
    B, G = len(lens), Hq // Hkv
    k, v, table = R.make_pool(lens, ps, Hkv, D, dt, seed=111)
    q = (torch.randn(B, Hq, D, generator=torch.Generator().manual_seed(112)) * 2).to(dt)
    got, lse, status = run_attention(k, v, table, lens, q)
    assert status == H.OK
    total = sum(max(1, -(-n // 64)) for n in lens) * Hkv
    share = -(-total // min(148, total))
    missed = places = 0
    for b, n in enumerate(lens):
        if n == 0:
            assert (got[b] == 0).all()
            continue
        pos = torch.arange(n)
        page = table[b].long()[pos // ps]
        parts = min(148, -(-(-(-n // 64)) // max(1, share - 1)) + 1)
        for h in range(Hkv):
            kk, vv = k[page, h, pos % ps].double(), v[page, h, pos % ps].double()
            qq = q[b, h * G:(h + 1) * G].double()
            x = qq @ kk.T * D ** -0.5
            rl = torch.logsumexp(x, -1)
            p = torch.exp(x - rl[:, None])
            out, size = p @ vv, p @ vv.abs()
            d = (2 * D + 8) * U * (qq.abs() @ kk.abs().T).amax(-1, keepdim=True) * D ** -0.5
            c = 2 * d + 2 * (4 * share + 3 * (10 + parts)) * U + 8 * U
            c = c + half_step(dt) ** (3 if dt == torch.bfloat16 else 2)
            bound = c * size + U * out.abs()
            if dt == torch.float16:
                bound = bound + 2.0 ** -40 * p.amax(-1, keepdim=True) * vv.abs().sum(0)
            err = (got[b, h * G:(h + 1) * G].double() - out).abs()
            assert (err <= bound).all(), f"{b} {h}: worst {float((err / bound).max()):.3f} of the bound"
            assert ((lse[b, h * G:(h + 1) * G].double() - rl).abs() <= c[:, 0] + 4 * U * rl.abs()).all()
            if n >= 64 * 8 and h == 0:     # what leaving out one tile would do
                for t in range(0, n // 64, max(1, n // 640)):
                    cut = slice(64 * t, 64 * t + 64)
                    less = (out - p[:, cut] @ vv[cut]) / (1 - p[:, cut].sum(-1, keepdim=True)).clamp(min=1e-30)
                    places += 1
                    missed += bool(((less - out).abs() <= bound).all())
    assert missed == 0, f"{missed} of {places} lost tiles would pass"


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 8, 1), (64, 12, 1), (128, 4, 2), (128, 16, 1)])
def test_third_part_of_bf16_probabilities(D, Hq, Hkv):
    """Two keys per sequence: weight 1 with value 0, weight p with value 1, so the output is
    p / (1 + p) and the rounding of p shows in full.  One channel makes the scores: the products
    are exact, x = s c has 3 u of |x| (c, the product, the maximum's subtraction), ex2.approx 4 u; the
    sum 1 + p, the division's two steps, the merges by factors of 1 and the parts' sums 10 u; three
    parts leave u16^3.  Two parts would leave up to u16^2 = 2^-16 and exceed the bound (checked on
    the reference)."""
    dt, ps, B = torch.bfloat16, 16, 96
    lens = [2] * B
    k, v, table = R.make_pool(lens, ps, Hkv, D, dt, seed=113)
    page = table[:, 0].long()
    g = torch.Generator().manual_seed(114)
    k[page, :, :2] = 0
    k[page, :, 0, 0] = 1
    s = -torch.rand(B, Hkv, generator=g).to(dt)                 # p between 1/e and 1, by scale 1
    k[page, :, 1, 0] = 1 + s
    s = k[page, :, 1, 0].double() - 1                           # what bf16 holds
    v[page, :, 0] = 0
    v[page, :, 1] = 1
    q = torch.zeros(B, Hq, D, dtype=dt)
    q[..., 0] = torch.linspace(0.5, 1, Hq).to(dt)
    got, _, status = run_attention(k, v, table, lens, q, scale=1.0)
    assert status == H.OK
    qs = q[..., 0].double()
    x = qs * s.repeat_interleave(Hq // Hkv, 1)                  # log of p
    p = x.exp()
    want = (p / (1 + p))[..., None].expand_as(got)
    c = (3 * 2 * U * (qs.abs() * 2) * 1.4427 + 4 * U + 10 * U + half_step(dt) ** 3)[..., None]
    assert ((got.double() - want).abs() <= c * want).all()
    hi = p.to(dt).double()
    lost = (p - hi - (p - hi).to(dt).double()).abs() / (1 + p)
    assert (lost[..., None] > 2 * c * want).any(-1).sum() > B * Hq // 8


@pytest.mark.parametrize("Hq,Hkv,D,ps,dt,src", [(25, 5, 64, 64, torch.float16, torch.float32),
                                                (32, 8, 128, 16, torch.bfloat16, torch.bfloat16),
                                                (16, 1, 128, 32, torch.float16, torch.float16)])
@pytest.mark.parametrize("step", [False, True])
def test_append_of_queries_only(Hq, Hkv, D, ps, dt, src, step):
    """A layer that reads another layer's cache rotates its queries and stores nothing: one token
    each and ragged rows; the cache may have no pool, the table no page."""
    start = [0, 5, ps - 1, 1000, 3, 2 ** 20]
    new = [1] * 6 if step else [3, 0, 2 * ps + 1, 1, ps, 70]
    T = sum(new)
    g = torch.Generator().manual_seed(115)
    wide = (torch.randn(T + 2, Hq * D + 64, generator=g) * 1.5).to(src)
    rows = wide[:T] if step else wide
    q = rows[:, 32:32 + Hq * D].unflatten(1, (Hq, D))
    pool = torch.full((3, Hkv, ps, D), 3.0, dtype=dt, device="cuda")
    bounds = torch.full((3, Hkv, D), 2.0, dtype=dt, device="cuda")
    cache = H.PagedCache(pool, pool.clone(), bounds, bounds.clone())
    table = torch.full((6, 2), -1, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    cu = [sum(new[:i]) for i in range(7)]
    dev = rows.cuda()[:, 32:32 + Hq * D].unflatten(1, (Hq, D))
    ws = H.alloc_workspace(256)
    outs = []
    for null in (False, True):
        if null:
            cache.c.k = cache.c.v = None
        out = torch.full((rows.shape[0], Hq, D), 5.0, dtype=dt, device="cuda")
        H.paged_append(cache, table, i32(start), None, None, ws, q=dev, q_out=out, cu_new=None if step else i32(cu))
        assert H.status_read(ws) == H.OK
        outs.append(out.cpu())
    assert torch.equal(*outs)
    for b in range(6):
        r = slice(cu[b], cu[b + 1])
        ref = R.rotate(q[r], list(range(start[b], start[b] + new[b])), 10000.0)
        mag = q[r].double().abs()
        mag = mag + torch.roll(mag, D // 2, -1)
        sub = 2.0 ** -25 if dt == torch.float16 else 0.0
        assert ((outs[0][r].double() - ref).abs() <= 8 * U * mag + half_step(dt) * ref.abs() + sub).all()
    assert (outs[0][cu[6]:] == 5).all()
    assert (pool == 3).all() and (cache.t["v"] == 3).all() and (bounds == 2).all()
