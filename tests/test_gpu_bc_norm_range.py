"""The norm of B and C of rows whose squares leave float32."""
import pytest
import torch

import delta_ref as ref
import ssd_chunked_scan_03_amd as ssd
from test_gpu_bc_norm import B16, F32, close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("N,F,mode", [(16, 4, "rms"), (128, 64, "l2"), (256, 0, "rms")])
def test_rows_whose_squares_overflow(N, F, mode, dtype):
    """Rows of 1 to 10^34 side by side, the values of each within two orders: the squares' sum is
    infinite in float32 from 10^19 on, the row's norm and its result are not.  Tolerances as in
    test_gpu_bc_norm."""
    g = torch.Generator().manual_seed(61)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    size = 10.0 ** torch.tensor([0.0, 18.0, 19.5, 25.0, 34.0, 3.0, 30.0]).view(1, -1, 1, 1)
    draw = lambda: (torch.randn(1, 7, 3, N, generator=g).double() * size).float().to(td)  # noqa: E731
    B, C = draw(), draw()
    dBn, dCn = (torch.randn(1, 7, 3, N, generator=g).to(td) for _ in range(2))
    w = 1 + 0.1 * torch.randn(N, generator=g)
    freq = (100.0 ** (-torch.arange(F) / max(F, 1))).float() if F else None
    pos = torch.arange(7, dtype=torch.int32)[None]
    dev = lambda v: None if v is None else v.cuda()  # noqa: E731
    kw = dict(mode=mode, inv_freq=dev(freq))
    Bn, Cn = ssd.bc_norm(B.cuda(), C.cuda(), w.cuda(), None, **kw)
    for got, v, wt in ((Bn, B, w), (Cn, C, None)):
        close(got, ref.norm(v, wt, mode, 1e-6, freq, pos, False), dtype, 24, (N, mode))
    out = ssd.bc_norm_bwd(B.cuda(), C.cuda(), dBn.cuda(), dCn.cuda(), w.cuda(), None, **kw)
    for n, dv, v, wt in (("dB", dBn, B, w), ("dC", dCn, C, None)):
        f = v.double().clone().requires_grad_()
        y = ref.norm(f, wt, mode, 1e-6, freq, pos, False)
        want, = torch.autograd.grad((y * dv.double()).sum(), [f])
        r = 1 / torch.sqrt(f.detach().square().sum(-1, keepdim=True) / (N if mode == "rms" else 1) + 1e-6)
        top = r * dv.double().abs().amax(-1, keepdim=True) * (1 if wt is None else wt.double().abs().max()) * 2
        got = out[n].double().cpu()
        lim = (B16 if dtype == "bf16" else F32) * want.abs() + 48 * F32 * (want.abs() + top)
        assert torch.isfinite(got).all() and ((got - want).abs() / lim).max().item() <= 1.0, (n, N, mode)
