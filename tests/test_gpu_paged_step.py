"""The mixer's decode step over pages with a ranked selection, and over bf16 pools, against the
fp64 oracle's layer whose attention is restricted to the positions that the definition of the
selection gives."""
import numpy as np
import pytest
import torch

from hybrid_attention_ssm_b200 import hymba as H
from hybrid_attention_ssm_b200 import synth
from oracle import hymba_oracle as orc
from tests import paged_ref as R
from tests.helpers import BF16_TOL, assert_rms, to_np
from tests.test_gpu_paged_mixer import paged_from, paged_step
from tests.test_gpu_parity import _ragged_case, _w

pytestmark = pytest.mark.gpu
WL = synth.workloads()


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    H.lib()


def projections(dims, w, st, positions):
    """Rotated query, rotated key and value of the new tokens, 64 bits: [B, heads, D] each."""
    proj = np.asarray(st["x_new"], np.float64) @ np.asarray(w["w_in"], np.float64).T
    q, k, v, _, _ = orc.split_in_proj(proj, dims)
    rot = lambda a, h: np.concatenate([orc.rope(a[b].reshape(1, 1, h, dims.head_dim), [p], dims.rope_base)[:, 0]
                                       for b, p in enumerate(positions)])
    t = torch.from_numpy
    return (t(rot(q, dims.n_q_heads)), t(rot(k, dims.n_kv_heads)),
            t(v.reshape(len(positions), dims.n_kv_heads, dims.head_dim)))


def layer_output(dims, w, st, positions, k, v, table, q, lists=None):
    """The oracle's layer with the attention over the pool's listed pages (or over what is visible)."""
    M, W = (0, 0) if dims.is_global else (dims.n_meta, dims.window)
    O, _, _ = R.attention(k, v, table, [p + 1 for p in positions], q, dims.head_dim ** -0.5, M, W, lists)
    outs = []
    for b, p in enumerate(positions):
        n = {"k": (1, p + 1), "v": (1, p + 1)} if dims.is_global else \
            {"meta_k": (1, dims.n_meta), "meta_v": (1, dims.n_meta), "ring_k": (1, dims.window), "ring_v": (1, dims.window)}
        cache = {a: np.zeros(s + (dims.n_kv_heads, dims.head_dim)) for a, s in n.items()}   # (its attention is not used)
        r = orc.mixer_decode(dims, w, st["x_new"][b:b + 1], p, cache, st["ssm_state"][b:b + 1], st["conv_state"][b:b + 1])
        outs.append(orc.fuse_and_project(O[b].reshape(1, -1).numpy(), r["y_ssm"], w, dims, None)[0][0])
    return np.stack(outs)


def chosen_pages(dims, lo, hi, table, positions, q, ps, top, u16):
    """The lists by the definition, after checking that no rounding of q can change them: u16 of
    each |q_d| against the largest bound, for the last page taken and the first one left out."""
    first = -(-dims.n_meta // ps)
    G = dims.n_q_heads // dims.n_kv_heads
    lists = torch.full((len(positions), dims.n_kv_heads, top), -1, dtype=torch.int32)
    for b, p in enumerate(positions):
        n = p // ps + 1
        sc = R.scores(lo, hi, table[b, :n], q[b])
        rows = table[b, :n].long()
        wide = torch.maximum(lo[rows].double().abs(), hi[rows].double().abs()).transpose(0, 1)   # [Hkv, n, D]
        slack = 2 * u16 * torch.einsum("ghd,gnd->gn", q[b].abs().view(dims.n_kv_heads, G, -1), wide)
        for h in range(dims.n_kv_heads):
            pick = R.select(sc[h].tolist(), first, 1, top)
            lists[b, h] = torch.tensor(pick, dtype=torch.int32)
            if n > top:
                free = [j for j in range(first, n - 1)]
                inside = [j for j in free if j in pick]
                outside = [j for j in free if j not in pick]
                assert min(sc[h, j] - slack[h, j] for j in inside) > max(sc[h, j] + slack[h, j] for j in outside)
    return lists


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("ps,top", [(16, 5), (32, 4)])
def test_step_attends_to_the_selected_pages(dt, ps, top):
    """Each sequence and kv head has its own few heavy pages (keys twice as large), so the ranking
    is clear of rounding; the step's output is the oracle's over exactly the listed pages: the
    meta tokens' page, the last one, and the heavy ones.  Any one page exchanged for one that is
    not listed would show (checked on the oracle).  A sequence begins a new page, one has no more pages than are
    read.  The query is rounded to the pool's type in the reference as in the kernel."""
    dims = WL["tiny"].dims.replace(is_global=1)
    positions = [dims.n_meta, 300, 159, 160, 411]
    B, Hkv, D = len(positions), dims.n_kv_heads, dims.head_dim
    w = _w(dims, seed=121)
    st, cache = _ragged_case(dims, B, positions, seed=122, Lmax=max(positions) + 1)
    rng = np.random.default_rng(123)
    for b, p in enumerate(positions):
        last = p // ps
        for h in range(Hkv):
            for j in rng.permutation(np.arange(1, max(last, 1)))[:top - 2]:
                cache["k"][b, j * ps:(j + 1) * ps, h] *= 2
    pc, table = paged_from(dims, cache, positions, ps, dtype=dt, bounds=True)
    out, _ = paged_step(dims, w, st, positions, pc, table, top=top)
    k, v, lo, hi = (pc.t[n].cpu() for n in ("k", "v", "k_lo", "k_hi"))
    tb = table.cpu()
    q, kn, vn = projections(dims, w, st, positions)
    u16 = torch.finfo(dt).eps / 2
    for b, p in enumerate(positions):     # the new token's row, which the reference takes from the pool
        assert_rms(k[tb[b, p // ps].long(), :, p % ps].double().numpy(), kn[b].numpy(), name=f"k row {b}")
        assert_rms(v[tb[b, p // ps].long(), :, p % ps].double().numpy(), vn[b].numpy(), name=f"v row {b}")
    lists = chosen_pages(dims, lo, hi, tb, positions, q, ps, top, u16)
    q = q.to(dt)
    want = layer_output(dims, w, st, positions, k, v, tb, q, lists)
    assert_rms(to_np(out), want, name=f"selected pages {dt} {ps}")
    rms = np.sqrt(np.mean(want * want))
    for b, p in enumerate(positions):
        if p // ps + 1 <= top:
            continue
        for h in range(Hkv):
            for i in range(top):
                other = lists.clone()
                other[b, h, i] = next(j for j in range(p // ps + 1) if j not in lists[b, h].tolist())
                off = layer_output(dims, w, st, positions, k, v, tb, q, other)
                assert np.abs(off[b] - want[b]).max() > 2 * BF16_TOL * rms, (b, h, i)


@pytest.mark.parametrize("ps", [16, 64])
@pytest.mark.parametrize("is_global", [0, 1])
def test_step_over_a_bf16_pool(is_global, ps):
    """Producer (or global) and consumer layers over bf16 pages: the oracle's attention over the
    pool's own rows, with the query rounded as in the kernel."""
    dims = WL["tiny"].dims.replace(window=32, is_global=is_global,
                                   kv_role=synth.KV_OWN if is_global else synth.KV_PRODUCER)
    M, W = dims.n_meta, dims.window
    positions = [M, M + 5, M + W - 1, M + W, M + 3 * W + 7, M + 1]
    w = _w(dims, seed=124)
    st, cache = _ragged_case(dims, len(positions), positions, seed=125, Lmax=max(positions) + 1 if is_global else 1)
    pc, table = paged_from(dims, cache, positions, ps, dtype=torch.bfloat16)
    layers = [(dims, w, st)]
    if not is_global:
        cons = dims.replace(kv_role=synth.KV_CONSUMER)
        layers.append((cons, _w(cons, seed=126), _ragged_case(cons, len(positions), positions, seed=127)[0]))
    for i, (dm, wt, state) in enumerate(layers):
        out, _ = paged_step(dm, wt, state, positions, pc, table)
        k, v, tb = pc.t["k"].cpu(), pc.t["v"].cpu(), table.cpu()
        if i == 0:
            q, kn, vn = projections(dm, wt, state, positions)
            for b, p in enumerate(positions):
                row = tb[b, p // ps].long()
                assert_rms(k[row, :, p % ps].double().numpy(), kn[b].numpy(), name=f"k row {b}")
                assert_rms(v[row, :, p % ps].double().numpy(), vn[b].numpy(), name=f"v row {b}")
        else:
            proj = np.asarray(state["x_new"], np.float64) @ np.asarray(wt["w_in"], np.float64).T
            qf = orc.split_in_proj(proj, dm)[0].reshape(len(positions), 1, 1, dm.n_q_heads, dm.head_dim)
            q = torch.from_numpy(np.concatenate([orc.rope(qf[b], [p], dm.rope_base)[:, 0]
                                                 for b, p in enumerate(positions)]))
        want = layer_output(dm, wt, state, positions, k, v, tb, q.to(torch.bfloat16))
        assert_rms(to_np(out), want, name=f"bf16 pool, layer {i}")
