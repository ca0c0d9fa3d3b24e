"""The mixer's decode step over a paged cache: against the fp64 oracle at each sequence's own
position, against the step over contiguous caches, and after a prefill whose cache rows were
moved into pages."""
import math

import numpy as np
import pytest
import torch

from hybrid_attention_ssm_b200 import hymba as H
from hybrid_attention_ssm_b200 import synth
from oracle import hymba_oracle as orc
from tests.helpers import PrefillRun, assert_elem, assert_rel_inf, assert_rms, bf16_dev, f32_dev, to_np
from tests.test_gpu_parity import _ragged_case, _ragged_oracle, _ragged_run, _w

pytestmark = pytest.mark.gpu
WL = synth.workloads()


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.lib()


def paged_from(dims, cache, positions, ps, dtype=torch.float16, seed=0, bounds=False):
    """A pool that holds what the contiguous caches hold before the step: all positions of a
    global layer, the meta tokens and the window of an SWA layer; NaN elsewhere, and no page
    where a whole page is hidden.  The new token's page is in the table."""
    B, M, W = len(positions), dims.n_meta, dims.window
    Hkv, D = dims.n_kv_heads, dims.head_dim
    width = max(positions) // ps + 1
    g = torch.Generator().manual_seed(seed)
    k = torch.full((B * width + 2, Hkv, ps, D), math.nan, dtype=dtype)
    v = k.clone()
    perm = torch.randperm(B * width + 2, generator=g)
    table = torch.full((B, width), -1, dtype=torch.int32)
    at = 0
    for b, p in enumerate(positions):
        for j in range(p // ps + 1):
            pos = [q for q in range(j * ps, min(p + 1, (j + 1) * ps))
                   if dims.is_global or q < M or p - q < W]
            if not pos:
                continue
            page = int(perm[at])
            at += 1
            table[b, j] = page
            for q in pos:
                if q == p:
                    continue
                for pool, n in ((k, "k"), (v, "v")):
                    row = (cache[n][b, q] if dims.is_global else
                           cache["meta_" + n][b, q] if q < M else cache["ring_" + n][b, (q - M) % W])
                    pool[page, :, q % ps] = torch.from_numpy(np.ascontiguousarray(row)).to(dtype)
    dev = [t.cuda() for t in (k, v)]
    if bounds:
        fill = torch.nan_to_num(dev[0].float(), nan=0.0)
        seen = ~torch.isnan(dev[0])
        dev.append(torch.where(seen, fill, math.inf).amin(2).to(dtype))
        dev.append(torch.where(seen, fill, -math.inf).amax(2).to(dtype))
    return H.PagedCache(*dev), table.cuda()


def paged_step(dims, w, st, positions, pc, table, top=0, ws=None):
    B = len(positions)
    ssm, conv = f32_dev(st["ssm_state"]), f32_dev(st["conv_state"])
    out = torch.zeros(B, dims.d_model, dtype=torch.bfloat16, device="cuda")
    ws = H.alloc_workspace(H.mixer_paged_workspace_size(dims, B, top)) if ws is None else ws
    pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
    H.mixer_decode_paged(dims, H.DeviceWeights(w), bf16_dev(st["x_new"]), pos, pc, table, ssm, conv, out, ws,
                         top_pages=top)
    torch.cuda.synchronize()
    assert H.status_read(ws) == 0
    return out, ssm


@pytest.mark.parametrize("ps", [16, 64])
@pytest.mark.parametrize("is_global", [0, 1])
def test_paged_decode_matches_the_oracle(is_global, ps):
    dims = WL["tiny"].dims.replace(window=32, is_global=is_global,
                                   kv_role=synth.KV_OWN if is_global else synth.KV_PRODUCER)
    M, W = dims.n_meta, dims.window
    positions = [M, M + 5, M + W - 1, M + W, M + 3 * W + 7, M + 1]
    Lmax = max(positions) + 1 if is_global else 1
    w = _w(dims, seed=41)
    st, cache = _ragged_case(dims, len(positions), positions, seed=42, Lmax=Lmax)
    pc, table = paged_from(dims, cache, positions, ps)
    out, ssm = paged_step(dims, w, st, positions, pc, table)
    ref_out, ref_state, ref_cache = _ragged_oracle(dims, w, st, cache, positions)
    assert_rms(to_np(out), ref_out, name="paged decode out")
    assert_rel_inf(to_np(ssm), ref_state, tol=1e-3, name="paged decode ssm state")
    for b, p in enumerate(positions):
        got = to_np(pc.t["k"][int(table[b, p // ps]), :, p % ps])
        want = ref_cache["k"][b, p] if is_global else ref_cache["ring_k"][b, orc.ring_slot(p, M, W)]
        assert_rms(got, want, name=f"k row (b={b})")
    if not is_global:   # the consumer of the pair reads the pages its producer appended to
        cons = dims.replace(kv_role=synth.KV_CONSUMER)
        wc = _w(cons, seed=43)
        stc, _ = _ragged_case(cons, len(positions), positions, seed=44)
        before = pc.t["k"].clone()
        outc, _ = paged_step(cons, wc, stc, positions, pc, table)
        refc, _, _ = _ragged_oracle(cons, wc, stc, ref_cache, positions)
        assert_rms(to_np(outc), refc, name="paged decode consumer out")
        assert torch.equal(before.view(torch.int16), pc.t["k"].view(torch.int16))


def test_paged_decode_hymba_width_equals_the_contiguous_step():
    """Hymba-width SWA layer: the paged step against the oracle, and against the step over the
    ring, whose sums run in another order.

    Two bf16 outputs of nearly equal values may be rounded to neighbours, a whole step apart:
    2^-7 |out| (2 half steps of 2^-8), which at |out| in [2, 4) is 1.6e-2, above 2e-2 of an
    RMS of 0.69.  Before that rounding the two differ by the fp16 roundings of the
    probabilities, the queries and u (2^-11 each, relative to terms that add up to about the
    RMS): 3 * 2^-11 = 1.5e-3 of the RMS, taken three times over."""
    wl = WL["decode_pair"]
    dims = wl.dims
    rng = np.random.default_rng(46)
    positions = sorted(int(v) for v in rng.integers(dims.n_meta, dims.n_meta + 4000, size=6)) + [dims.n_meta, 1151]
    w = _w(dims, wl=wl, layer=3)
    st, cache = _ragged_case(dims, len(positions), positions, seed=47)
    pc, table = paged_from(dims, cache, positions, 64)
    out, ssm = paged_step(dims, w, st, positions, pc, table)
    out_r, ssm_r, _, _ = _ragged_run(dims, w, st, cache, positions, 1)
    ref_out, _, _ = _ragged_oracle(dims, w, st, cache, positions)
    assert_rms(to_np(out), ref_out, name="paged decode out (Hymba width)")
    assert_elem(to_np(out), to_np(out_r), rel=2.0 ** -7, abs_rms=4.5e-3, name="paged against contiguous")
    assert torch.equal(ssm, ssm_r)


def test_paged_decode_page_selection():
    """Selecting as many pages as there are is attending to all of them, bit for bit; selecting
    fewer equals the layer over exactly those pages (bf16 pool)."""
    dims = WL["tiny"].dims.replace(is_global=1)
    positions = [dims.n_meta, 300, 159, 160]
    w = _w(dims, seed=51)
    st, cache = _ragged_case(dims, 4, positions, seed=52, Lmax=301)
    runs = {}
    for top in (0, 19, 6):
        pc, table = paged_from(dims, cache, positions, 16, dtype=torch.bfloat16, bounds=True)
        runs[top] = paged_step(dims, w, st, positions, pc, table, top=top)[0]
    assert torch.equal(runs[0], runs[19])
    # 160 and 159: 11 and 10 pages, of which 6 are read; position n_meta has one page
    assert torch.equal(runs[6][0], runs[0][0]) and not torch.equal(runs[6][1], runs[0][1])


def test_prefill_then_paged_steps():
    """A prefill's contiguous cache rows moved into pages (append without rotation), then decode
    steps over the pages beside the steps over the contiguous cache, on one workspace that other
    decode calls use in between, and once from a captured graph."""
    dims = WL["tiny"].dims.replace(is_global=1)
    B, N, steps, ps = 2, 70, 3, 32
    w = _w(dims, seed=61)
    rng = np.random.default_rng(62)
    X = synth.bf16_round(rng.normal(size=(B, N + steps, dims.d_model)).astype(np.float32))
    T = dims.n_meta + N
    run = PrefillRun(dims, w, X[:, :N], max_tokens=T + steps)
    ref = orc.mixer_prefill(dims, w, X)
    width = (T + steps) // ps + 1
    pc = H.PagedCache.zeros(B * width, ps, dims.n_kv_heads, dims.head_dim, bounds=True)
    table = torch.arange(B * width, dtype=torch.int32, device="cuda").flip(0).view(B, width)
    rows = lambda n: run.cache.t[n][:, :T].reshape(B * T, dims.n_kv_heads, dims.head_dim)
    need = max(H.mixer_paged_workspace_size(dims, B, 2), H.workspace_size(dims, B, T + steps, 0, H.MODE_DECODE))
    ws = H.alloc_workspace(need)
    H.paged_append(pc, table, torch.zeros(B, dtype=torch.int32, device="cuda"), rows("k"), rows("v"), ws,
                   cu_new=torch.tensor([0, T, 2 * T], dtype=torch.int32, device="cuda"), rope_base=0.0)
    for b in range(B):
        for n in ("k", "v"):
            got = pc.t[n][table[b].long()].transpose(1, 2).reshape(width * ps, dims.n_kv_heads, dims.head_dim)[:T]
            assert torch.equal(got, run.cache.t[n][b, :T])
    ssm, conv = [run.ssm.clone() for _ in range(2)], [run.conv.clone() for _ in range(2)]
    out = [torch.zeros(B, dims.d_model, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    x = torch.zeros(B, dims.d_model, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(B, dtype=torch.int32, device="cuda")
    graph = None
    for i in range(steps):
        x.copy_(bf16_dev(X[:, N + i]))
        pos.fill_(T + i)
        H.mixer_decode(dims, run.dw, x, T + i, run.cache, ssm[0], conv[0], out[0], ws)
        if i == 0:
            H.mixer_decode_paged(dims, run.dw, x, pos, pc, table, ssm[1], conv[1], out[1], ws)
        elif graph is None:
            graph = torch.cuda.CUDAGraph()
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
                H.mixer_decode_paged(dims, run.dw, x, pos, pc, table, ssm[1], conv[1], out[1], ws)
            torch.cuda.synchronize()
        if graph is not None:
            graph.replay()
        torch.cuda.synchronize()
        assert H.status_read(ws) == 0
        assert_rms(to_np(out[1]), ref["out"][:, T + i], name=f"paged step {i}")
        assert_rms(to_np(out[0]), ref["out"][:, T + i], name=f"contiguous step {i}")


def test_paged_decode_refusals():
    dims = WL["tiny"].dims
    B = 2
    w = H.DeviceWeights(_w(dims, seed=71))
    x = torch.zeros(B, dims.d_model, dtype=torch.bfloat16, device="cuda")
    pos = torch.full((B,), dims.n_meta, dtype=torch.int32, device="cuda")
    pc = H.PagedCache.zeros(8, 16, dims.n_kv_heads, dims.head_dim)
    table = torch.arange(8, dtype=torch.int32, device="cuda").view(2, 4)
    ssm, conv = torch.zeros(B, dims.d_inner, 16, device="cuda"), torch.zeros(B, dims.d_inner, 3, device="cuda")
    ws = H.alloc_workspace(H.mixer_paged_workspace_size(dims, B))
    good = dict(dims=dims, dw=w, x=x, positions=pos, cache=pc, table=table, ssm_state=ssm, conv_state=conv,
                out=torch.zeros_like(x), ws=ws)
    H.mixer_decode_paged(**good)
    assert H.status_read(ws) == 0
    wide = H.PagedCache.zeros(8, 16, dims.n_kv_heads, 128)
    heads = H.PagedCache.zeros(8, 16, dims.n_kv_heads + 1, dims.head_dim)
    for bad in (dict(positions=pos.long()), dict(positions=pos[:1]), dict(cache=wide), dict(cache=heads),
                dict(top_pages=2), dict(top_pages=-1), dict(dims=dims.replace(is_global=1), top_pages=2),
                dict(ws=ws[:1024]), dict(x=x[:1]), dict(out=torch.zeros(B, 8, dtype=torch.bfloat16, device="cuda"))):
        with pytest.raises(H.HymbaError):
            H.mixer_decode_paged(**{**good, **bad})
    pos.fill_(64)   # beyond the table: recorded
    H.mixer_decode_paged(**good)
    assert H.status_read(ws) == H.ERR_INVALID_ARG
