"""ssv_logprobs over rows of every kind at once against torch in 64 bits, whatever number of CTAs, threads and
candidates a row takes: few and many alternatives beside few and many elements (tolerances: logits_common)."""
import numpy as np
import pytest
import torch

from diffusion_speculative_verification_gb300 import ssv
from gpu_common import ensure_built
from logits_common import EPS, LN, near

pytestmark = pytest.mark.gpu


def setup_module():
    ensure_built()


@pytest.mark.parametrize("v", [130, 255, 520, 777, 1024, 2048, 4001, 6000, 16384, 100003])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n", [1, 20, 500])
def test_alternatives(n, dtype, v):
    g = torch.Generator(device="cuda").manual_seed(v + n)
    x = (torch.randn(n, v, generator=g, device="cuda") * 2).to(dtype)
    x[n // 2, : v // 2] = x[n // 2, v // 2].clone()                   # a run of equal logits
    tok = torch.randint(0, v, (n,), generator=g, device="cuda").int()
    lp = torch.log_softmax(x.double(), 1)
    order = torch.sort(x.float(), dim=1, descending=True, stable=True).indices
    rank = (order == tok[:, None]).int().argmax(1) + 1
    ent = -(lp.exp() * lp).sum(1)
    for k in (1, 33, 64, 65, 100, 128):
        logprob, r, e, lse, tl, tt = ssv.logprobs(x, tok, k)
        c = min(k, v)
        assert torch.equal(tt[:, :c].long(), order[:, :c]) and (tt[:, c:] == -1).all()
        assert torch.equal(r.long(), rank)
        want = lp.gather(1, order[:, :c]).cpu().numpy()
        near(tl[:, :c].cpu().numpy(), want, LN + 4 * EPS * np.abs(want))
        want = lp.gather(1, tok.long()[:, None])[:, 0].cpu().numpy()
        near(logprob.cpu().numpy(), want, LN + EPS * np.abs(want))
        near(e.cpu().numpy(), ent.cpu().numpy(), 2 * LN * (1 + ent.abs().cpu().numpy()))
