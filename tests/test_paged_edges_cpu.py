"""More refusals of the paged calls, decided on the host (the made-up addresses of
test_paged_cpu are never touched)."""
import ctypes
import types

import pytest
import torch

from hybrid_attention_ssm_b200 import build as hbuild
from hybrid_attention_ssm_b200 import hymba as H
from hybrid_attention_ssm_b200 import synth
from tests.test_paged_cpu import A, append


@pytest.fixture(scope="module", autouse=True)
def _lib():
    hbuild.build()
    H.lib()


def test_queries_in_place_need_the_rows_of_the_output():
    """q_out may be q itself only where a row of one is a row of the other: wider source elements
    or a larger row stride would let one token's result overwrite another's query."""
    for kw in (dict(src=H.DT_F32), dict(src=H.DT_BF16), dict(src=H.DT_F16, qs=264), dict(src=H.DT_F16, qs=512, cu=None)):
        assert append(**{**dict(q=A, q_out=A), **kw}) == H.ERR_INVALID_ARG, kw


def test_mixer_step_refuses_tensors_that_the_kernels_would_misread(monkeypatch):
    """Types, sizes and contiguity of everything that the layer's step reads or writes.  The
    tensors are on the host, so the device checks are stood in for; a call that passes the
    binding's checks ends in a stub."""
    dims = synth.workloads()["tiny"].dims
    B, d, Di = 2, dims.d_model, dims.d_inner
    reached = []

    class Lib:
        def hymba_mixer_decode_paged(self, *a):
            reached.append(a)
            return H.OK

    pool = torch.zeros(8, dims.n_kv_heads, 16, dims.head_dim, dtype=torch.float16)
    pc = H.PagedCache.__new__(H.PagedCache)
    pc.t, pc.device, pc.dtype, pc.n_kv_heads, pc.head_dim = {"k": pool}, -1, pool.dtype, dims.n_kv_heads, dims.head_dim
    pc.c = H.PagedKV()
    pc.ref = ctypes.byref(pc.c)
    dw = types.SimpleNamespace(c=H.LayerWeights())
    monkeypatch.setattr(H, "lib", lambda: Lib())
    monkeypatch.setattr(H, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
    good = dict(dims=dims, dw=dw, x=bf(B, d), positions=torch.zeros(B, dtype=torch.int32), cache=pc,
                table=torch.zeros(B, 4, dtype=torch.int32), ssm_state=torch.zeros(B, Di, 16),
                conv_state=torch.zeros(B, Di, 3), out=bf(B, d), ws=torch.zeros(1024, dtype=torch.uint8),
                residual=bf(B, d))
    H.mixer_decode_paged(**good)
    H.mixer_decode_paged(**{**good, "residual": None})
    H.mixer_decode_paged(**{**good, "ssm_state": torch.zeros(B + 3, Di, 16)})   # states of a larger batch
    assert len(reached) == 3
    for bad in (dict(x=torch.zeros(B, d)), dict(x=torch.zeros(B, d, dtype=torch.float16)), dict(out=torch.zeros(B, d)),
                dict(x=bf(B, 2 * d)[:, ::2]), dict(out=bf(2 * B, d)[::2]), dict(residual=torch.zeros(B, d)),
                dict(residual=bf(B - 1, d)), dict(residual=bf(d, B).T), dict(ssm_state=bf(B, Di, 16)),
                dict(ssm_state=torch.zeros(B, Di, 15)), dict(ssm_state=torch.zeros(B, 16, Di).transpose(1, 2)),
                dict(conv_state=torch.zeros(B, Di, 3, dtype=torch.float64)), dict(conv_state=torch.zeros(B - 1, Di, 3)),
                dict(conv_state=torch.zeros(B, Di, 4)[..., :3])):
        with pytest.raises(H.HymbaError):
            H.mixer_decode_paged(**{**good, **bad})
    assert len(reached) == 3
