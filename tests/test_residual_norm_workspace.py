"""The workspace of the norms' backward: as large as it says, written nowhere else, and no
larger than its calls can use."""
import ctypes

import pytest
import torch

from grpo_loss_gb300 import _lib as L

F32, BF16 = torch.float32, torch.bfloat16
CODE = {F32: L.GRPO_F32, BF16: L.GRPO_BF16}


def size_of(rows, d, dtype, rms, gate_rows):
    return L.residual_norm_workspace_size(L.ResidualNormProblem(rows, d, *[0] * 10, gate_rows, 1e-5, 1.0, int(rms), CODE[dtype],
                                                                L.GRPO_F32, CODE[dtype]))


@pytest.mark.gpu
@pytest.mark.parametrize("gate", ["none", "shared", "some", "all"])
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dtype,rows,d", [(BF16, 9000, 64), (F32, 9000, 512), (BF16, 6000, 1000), (BF16, 4000, 1001), (F32, 3000, 1536), (BF16, 3000, 4096),
                                          (BF16, 2048, 4097), (BF16, 2500, 6144), (BF16, 2500, 8192), (BF16, 3000, 8191), (F32, 1200, 8192),
                                          (F32, 700, 8193), (BF16, 1500, 12288), (BF16, 900, 16384), (BF16, 600, 32768), (F32, 400, 32767)])
def test_nothing_behind_it_is_written(dtype, rows, d, rms, gate):
    import grpo_loss_gb300 as G
    g = torch.Generator(device="cuda").manual_seed(d)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, h, dy, dh = (n(rows, d).to(dtype) for _ in range(4))
    m, r, pm, pr = n(rows), 0.5 + n(rows).abs(), n(rows), 0.5 + n(rows).abs()
    gt = {"none": None, "shared": n(1, d), "some": n(next(k for k in range(rows // 100, 0, -1) if rows % k == 0), d), "all": n(rows, d)}[gate]
    gt = None if gt is None else gt.to(dtype)
    per = 0 if gt is None else rows // len(gt)
    size, guard = size_of(rows, d, dtype, rms, per), 1 << 16
    ws = torch.full((size + guard,), 0x5A, dtype=torch.uint8, device="cuda")
    for post in (False, True):
        kw = dict(x=x, gate=gt, rms=rms, bias=not rms, scale=0.5)
        if post:
            kw.update(post_weight=n(d), post_rstd=pr, post_mean=None if rms else pm, post_bias=None if rms else n(d))
        ws.fill_(0x5A)
        w = n(d).abs_()
        want = G.residual_norm_bwd(dy, dh, h, w, None if rms else m, r, **kw)
        got = G.residual_norm_bwd(dy, dh, h, w, None if rms else m, r, workspace=ws[:size], **kw)
        assert (ws[size:] == 0x5A).all()
        assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(want, got))
        if post and gate != "all":
            assert (ws[:size] != 0x5A).any()


@pytest.mark.gpu
def test_its_size():
    """Column sums of the parameters that there are, for as many walkers as an SM holds."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    for rows, d, each in ((1 << 20, 256, 32), (1 << 20, 4096, 8), (1 << 18, 8192, 4), (1 << 16, 32768, 2)):
        one = 4 * d * each * sms
        assert size_of(rows, d, BF16, True, 0) == 2 * one and size_of(rows, d, BF16, False, 1) == 4 * one
        assert size_of(rows, d, BF16, True, rows) == 4 * one and size_of(rows, d, BF16, False, 7) == 6 * one
        assert size_of(1, d, BF16, True, 0) == 2 * 4 * d * 8


@pytest.mark.gpu
def test_a_size_for_each_kind_of_call():
    """A call without a gate does not leave its size for one with."""
    import grpo_loss_gb300 as G
    rows, d = 1000, 320
    x, r, w = torch.randn(rows, d, device="cuda"), torch.ones(rows, device="cuda"), torch.ones(d, device="cuda")
    for rms in (True, False):
        for gate in (None, torch.ones(1, d, device="cuda"), torch.ones(rows, d, device="cuda"), torch.ones(10, d, device="cuda")):
            G.residual_norm_bwd(x, None, x, w, None if rms else r, r, x=x, gate=gate, rms=rms)
    size = ctypes.c_size_t(0)
    p = L.ResidualNormProblem(rows, d, *[0] * 10, 100, 1e-5, 1.0, 1, 0, 0, 0)
    assert L.lib().grpo_residual_norm_workspace_size(ctypes.byref(p), ctypes.byref(size)) == 0
    gate = torch.ones(10, d, device="cuda")
    with pytest.raises(L.GrpoError) as e:
        G.residual_norm_bwd(x, None, x, w, None, r, x=x, gate=gate, rms=True, workspace=torch.empty(size.value - 1, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 3
    G.residual_norm_bwd(x, None, x, w, None, r, x=x, gate=gate, rms=True, workspace=torch.empty(size.value, dtype=torch.uint8, device="cuda"))
