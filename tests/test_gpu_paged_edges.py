"""The paged cache operators at the ends of what their arguments may be, against the 64-bit
definitions in paged_ref; bounds as derived in test_gpu_paged."""
import threading

import pytest
import torch

from hybrid_attention_ssm_b200 import hymba as H
from tests import paged_ref as R
from tests.test_gpu_paged import check_attention, run_attention, run_select

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.lib()


@pytest.mark.parametrize("M", [2 ** 31 - 1, 2 ** 31 - 64, 2 ** 31 - 65])
@pytest.mark.parametrize("W", [5, 2 ** 31 - 1])
def test_meta_count_up_to_the_largest_int(M, W):
    """More meta tokens than any sequence has: every position is visible, whatever the window."""
    lens, ps, Hq, Hkv, D, dt = [0, 1, 5, 6, 64, 257, 3000], 32, 10, 2, 64, torch.float16
    k, v, table = R.make_pool(lens, ps, Hkv, D, dt, seed=90)
    q = torch.randn(len(lens), Hq, D, generator=torch.Generator().manual_seed(91)).to(dt)
    ref = R.attention(k, v, table, lens, q, D ** -0.5)
    got, lse, status = run_attention(k, v, table, lens, q, n_meta=M, window=W)
    assert status == H.OK
    check_attention(got, lse, ref, v, max(lens), dt, torch.float32, D)


def test_workspace_init_leaves_what_lies_behind_the_status():
    """hymba_workspace_init zeroes the status word's 256 bytes; a live workspace keeps the rest."""
    ws = H.alloc_workspace(8192)
    ws.fill_(0xa5)
    H.check(H.lib().hymba_workspace_init(H.ptr(ws), ws.numel(), H.stream_handle(None)))
    torch.cuda.synchronize()
    assert (ws[:256] == 0).all() and (ws[256:] == 0xa5).all()


def test_attention_after_other_calls_on_its_workspace():
    """Whatever other calls leave behind the status word, the attention joins the parts of a
    sequence that is cut over many CTAs; reading the status in between changes nothing."""
    lens, ps, Hq, Hkv, D, dt = [9000, 40], 64, 10, 2, 64, torch.float16
    k, v, table = R.make_pool(lens, ps, Hkv, D, dt, seed=92)
    cache = H.PagedCache(k.cuda(), v.cuda())
    q = torch.randn(2, Hq, D, generator=torch.Generator().manual_seed(93)).to(dt).cuda()
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ws = H.alloc_workspace(H.paged_workspace_size(cache, 2, Hq, table.shape[1]))
    want = torch.empty(2, Hq, D, device="cuda")
    H.paged_attention(cache, q, table.cuda(), ln, want, ws)
    assert H.status_read(ws) == H.OK
    for fill in (0xff, 0x01, 0x5a):
        ws[256:] = fill          # as any call may that keeps its buffers there
        got = torch.full_like(want, -7.0)
        H.paged_attention(cache, q, table.cuda(), ln, got, ws)
        assert H.status_read(ws) == H.OK
        assert torch.equal(got, want), hex(fill)
        assert (ws[:256] == 0).all()


@pytest.mark.parametrize("Hq,Hkv,D,dt", [(10, 2, 64, torch.float16), (12, 1, 64, torch.bfloat16),
                                         (4, 1, 128, torch.bfloat16), (16, 1, 128, torch.float16)])
def test_rows_whose_every_score_is_infinite(Hq, Hkv, D, dt):
    """Keys of -inf in channel 0: a head with a positive query there scores -inf everywhere and
    gets zeros and an lse of -inf, one with a negative query scores +inf and gets NaN; a head of
    query 0 in that channel has 0 * inf.  The other sequences are as without them.  One sequence
    within a tile, one cut over many CTAs."""
    lens, ps = [40, 20000, 0, 130], 64
    k, v, table = R.make_pool(lens, ps, Hkv, D, dt, seed=94)
    q = torch.randn(len(lens), Hq, D, generator=torch.Generator().manual_seed(95)).to(dt)
    q[:, :, 0] = 1.0
    q[:, 1, 0] = -1.0
    q[:, 2, 0] = 0.0
    want, wl, _ = run_attention(k, v, table, lens, q)
    for b in (0, 1):
        for j in range(-(-lens[b] // ps)):
            k[table[b, j], :, :, 0] = -float("inf")
    got, lse, status = run_attention(k, v, table, lens, q)
    assert status == H.OK
    low = [h for h in range(Hq) if h not in (1, 2)]
    assert (got[:2, low] == 0).all() and (lse[:2, low] == -float("inf")).all()
    assert got[:2, 1:3].isnan().all() and lse[:2, 1:3].isnan().all()
    assert torch.equal(got[2:], want[2:]) and torch.equal(lse[2:], wl[2:])


@pytest.mark.parametrize("B,Hkv,width", [(6, 5, 640), (12, 5, 640), (20, 5, 640), (45, 4, 640), (1, 2, 15000), (20, 1, 14001)])
def test_select_with_clusters_of_every_size(B, Hkv, width):
    """Numbers of lists and table widths between which the size of the cluster that serves a list
    changes; full and short lists side by side."""
    ps, D, dt, top = 16, 64, torch.float16, 24
    g = torch.Generator().manual_seed(96)
    n_pages = 700
    mid, wid = torch.randn(n_pages, Hkv, D, generator=g), torch.rand(n_pages, Hkv, D, generator=g)
    lo, hi = (mid - wid).to(dt), (mid + wid).to(dt)
    pages = [width if b % 2 == 0 else 1 + (width * b) // B for b in range(B)]
    table = torch.randint(0, n_pages, (B, width), generator=g).to(torch.int32)
    q = torch.randn(B, 2 * Hkv, D, generator=g).to(dt)
    got, status = run_select(lo, hi, table, [n * ps for n in pages], q, ps, top, 2, 1)
    assert status == H.OK
    for b, n in enumerate(pages):
        every = R.scores(lo, hi, torch.arange(n_pages), q[b])[:, table[b, :n].long()]
        for h in range(Hkv):
            assert got[b, h].tolist() == R.select(every[h].tolist(), 2, 1, top), (b, h)


def test_fp16_outputs_out_of_range_are_recorded():
    """A bf16 pool's values may lie beyond fp16: the output is infinite there, and the status says
    so; in the other types, and with values that fit, it stays clear."""
    dt = torch.bfloat16
    k, v, table = R.make_pool([40, 9000], 64, 2, 64, dt, seed=97)
    q = torch.randn(2, 10, 64, generator=torch.Generator().manual_seed(98)).to(dt)
    big = v.clone()
    big[table[0, 0].long(), 1, :, 7] = 1e5          # one channel of one kv head, in every row of its page
    for b in range(2):
        if b:                                       # and the same in the sequence that is cut and joined
            big[table[1, :141].long(), 1, :, 7] = 1e5
        got, _, status = run_attention(k, big, table, [40, 9000], q, torch.float16)
        assert status == H.ERR_FP16_RANGE
        for s in range(2):
            assert torch.equal(got[s].isinf(), (torch.zeros(10, 64) + (0 if s > b else 1)).bool() &
                               (torch.arange(10) >= 5)[:, None] & (torch.arange(64) == 7))
    for vals, out_dt in ((big, torch.bfloat16), (big, torch.float32), (v, torch.float16)):
        got, _, status = run_attention(k, vals, table, [40, 9000], q, out_dt)
        assert status == H.OK and got.isfinite().all()


def test_select_captured_and_from_several_threads():
    """A selection served by clusters, captured into a graph, and called from several host threads on
    streams and workspaces of their own: what the first eager call of a process asks CUDA about
    the device must not matter to either."""
    dt, D, Hkv, B, width, top = torch.bfloat16, 128, 4, 12, 700, 20
    g = torch.Generator().manual_seed(99)
    lo = torch.randn(800, Hkv, D, generator=g).to(dt)
    hi = lo + torch.rand(800, Hkv, D, generator=g).to(dt)
    k = torch.zeros(800, Hkv, 16, D, dtype=dt, device="cuda")
    cache = H.PagedCache(k, k, lo.cuda(), hi.cuda())
    table = torch.randint(0, 800, (B, width), generator=g).to(torch.int32)
    q = torch.randn(B, 8, D, generator=g).to(dt)
    lens = torch.full((B,), width * 16, dtype=torch.int32, device="cuda")
    tb, qg = table.cuda(), q.cuda()
    res = [torch.full((B, Hkv, top), 77, dtype=torch.int32, device="cuda") for _ in range(5)]
    wss = [H.alloc_workspace(256) for _ in range(5)]
    torch.cuda.synchronize()
    graph, st = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(st), torch.cuda.graph(graph, stream=st):
        H.paged_select(cache, qg, tb, lens, res[0], wss[0])
    graph.replay()
    errors = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            for _ in range(20):
                H.paged_select(cache, qg, tb, lens, res[i], wss[i], stream=s)
            s.synchronize()
        except Exception as e:   # a failure in a thread must reach the test
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(1, 5)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors and all(H.status_read(w) == H.OK for w in wss)
    for r in res[1:]:
        assert torch.equal(r, res[0])
    got = res[0].cpu()
    for b in range(B):
        sc = R.scores(lo, hi, table[b], q[b])
        for h in range(Hkv):
            assert got[b, h].tolist() == R.select(sc[h].tolist(), 1, 1, top)
