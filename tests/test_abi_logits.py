"""Host-side refusals of the logits operators (no GPU): bad arguments return synchronously, nothing is launched;
empty calls are no-ops."""
import ctypes as C

import pytest
import torch

from diffusion_speculative_verification_gb300 import build, ssv


@pytest.fixture(scope="module")
def L():
    build.build()
    return ssv.lib()


M = 1 << 24  # made-up addresses


def _logprobs(**kw):
    base = dict(logits=M, logits_stride=0, dtype=ssv.SSV_BF16, V=1000, total_rows=8, rows=None, tokens=2 * M, n=8, top_k=4,
                T=1.0, logprob=3 * M, rank=4 * M, entropy=5 * M, lse=6 * M, top_logprob=7 * M, top_token=8 * M,
                dev_status=None)
    base.update(kw)
    return ssv.LogprobsArgs(**base)


def test_logprobs_validation(L):
    inv = ssv.SSV_ERR_INVALID
    cases = [(dict(logits=None), inv), (dict(logits=M + 1), inv), (dict(dtype=ssv.SSV_F32, logits=M + 2), inv),
             (dict(dtype=2), inv), (dict(V=0), inv), (dict(V=(1 << 19) + 1), ssv.SSV_ERR_UNSUPPORTED),
             (dict(logits_stride=999), inv), (dict(logits_stride=-1000), inv), (dict(n=-1), inv), (dict(n=9), inv),
             (dict(total_rows=-1), inv), (dict(top_k=-1), inv), (dict(top_k=129), ssv.SSV_ERR_UNSUPPORTED),
             (dict(top_logprob=None), inv), (dict(top_token=None), inv), (dict(logprob=None), inv),
             (dict(tokens=None), inv), (dict(tokens=None, logprob=None), inv)]
    cases += [({k: a + 2}, inv) for k, a in (("tokens", 2 * M), ("rows", 9 * M), ("lse", 6 * M), ("top_token", 8 * M), ("rank", 4 * M))]
    cases += [(dict(lse=M + 100), inv), (dict(top_token=M + 2 * 8 * 1000 - 4), inv), (dict(logprob=M - 16), inv)]   # over the logits
    cases += [(dict(T=t), ssv.SSV_ERR_NOT_FINITE) for t in (0.0, -1.0, float("inf"), float("nan"), 1e-45)]
    cases += [(dict(tokens=None, logprob=None, rank=None, entropy=None, lse=None, top_k=0), inv)]  # nothing is asked for
    for kw, code in cases:
        assert L.ssv_logprobs(C.byref(_logprobs(**kw)), None) == code, kw
    assert L.ssv_logprobs(None, None) == inv
    assert L.ssv_logprobs(C.byref(_logprobs(n=0)), None) == ssv.SSV_OK


def _distill(**kw):
    base = dict(logits=M, logits_stride=0, dtype=ssv.SSV_BF16, V=1000, n=8, K=4, teacher_token=2 * M, teacher_logprob=3 * M,
                T=1.0, mode=ssv.REST, weight=4 * M, loss=5 * M, stats=6 * M, grad_loss=None, grad=7 * M, grad_stride=0,
                dev_status=None)
    base.update(kw)
    return ssv.DistillArgs(**base)


def test_distill_validation(L):
    inv = ssv.SSV_ERR_INVALID
    both = [(dict(logits=None), inv), (dict(logits=M + 1), inv), (dict(grad=7 * M + 1), inv), (dict(dtype=9), inv),
            (dict(V=0), inv), (dict(V=1 << 20), ssv.SSV_ERR_UNSUPPORTED), (dict(K=0), inv), (dict(K=129), ssv.SSV_ERR_UNSUPPORTED),
            (dict(n=-1), inv), (dict(mode=2), inv), (dict(logits_stride=500), inv), (dict(grad_stride=999), inv),
            (dict(teacher_token=None), inv), (dict(teacher_logprob=None), inv), (dict(T=0.0), ssv.SSV_ERR_NOT_FINITE),
            (dict(T=float("nan")), ssv.SSV_ERR_NOT_FINITE),
            (dict(teacher_token=2 * M + 1), inv), (dict(teacher_logprob=3 * M + 2), inv), (dict(weight=4 * M + 2), inv),
            (dict(stats=6 * M + 2), inv), (dict(loss=5 * M + 1), inv),
            # a gradient over logits that other CTAs still read
            (dict(grad=M + 32), inv), (dict(grad=M, grad_stride=1008), inv), (dict(grad=M - 32), inv),
            (dict(logits_stride=2000, grad_stride=2000, grad=M + 2 * 999), inv),
            (dict(logits_stride=2000, grad_stride=2000, grad=M + 2 * 1001), inv),
            (dict(grad=M + 2 * 7999), inv)]
    for kw, code in both:
        assert L.ssv_distill(C.byref(_distill(**kw)), None) == code, kw
        assert L.ssv_distill_backward(C.byref(_distill(**kw)), None) == code, kw
    for kw in (dict(loss=None), dict(grad_loss=8 * M), dict(loss=M + 64), dict(stats=M + 2 * 8 * 1000 - 16), dict(stats=7 * M),
               dict(loss=7 * M + 400)):
        assert L.ssv_distill(C.byref(_distill(**kw)), None) == inv, kw
    for kw in (dict(stats=None), dict(grad=None), dict(stats=7 * M + 256)):
        assert L.ssv_distill_backward(C.byref(_distill(**kw)), None) == inv, kw
    for f in (L.ssv_distill, L.ssv_distill_backward):
        assert f(None, None) == inv
        assert f(C.byref(_distill(n=0)), None) == ssv.SSV_OK


def refused(f, *a, match=None, **kw):
    with pytest.raises(ssv.SsvError, match=match) as e:
        f(*a, **kw)
    assert e.value.code == ssv.SSV_ERR_INVALID


def test_binding_refuses_wrong_tensors():
    """Shapes, types and strides are checked before any address is passed on."""
    x = torch.zeros((4, 10))
    tok = torch.zeros(4, dtype=torch.int32)
    refused(ssv.logprobs, x.half(), tok)
    refused(ssv.logprobs, x[0], tok)
    refused(ssv.logprobs, x.t(), tok)
    refused(ssv.logprobs, x[:1].expand(4, 10), tok)
    refused(ssv.logprobs, x, tok.long())
    refused(ssv.logprobs, x, tok[:, None])
    refused(ssv.logprobs, x, tok, rows=tok[:3])
    refused(ssv.logprobs, x, tok, rows=tok.long())
    refused(ssv.logprobs, x, tok, top_k=-1)
    f = torch.zeros(4)
    out = (f, tok, f, f, torch.zeros((4, 3)), torch.zeros((4, 3), dtype=torch.int32))
    for i, bad in enumerate((f[:3], f, f.double(), f[::2], torch.zeros((4, 4)), torch.zeros((4, 3)))):
        refused(ssv.logprobs, x, tok, 3, out=out[:i] + (bad,) + out[i + 1:])
    t, lp = torch.zeros((4, 3), dtype=torch.int32), torch.zeros((4, 3))
    for a in ((x, t.long(), lp), (x, t, lp.double()), (x, t[:3], lp[:3]), (x, t, lp[:, :2]), (x, t[:, 0], lp[:, 0]),
              (x.t(), t, lp), (x[0], t, lp), (x.double(), t, lp)):
        refused(ssv.distill, *a)
        refused(ssv.distill_backward, *a, torch.zeros((4, 4)))
    refused(ssv.distill, x, t, lp, weight=f[:3])
    refused(ssv.distill, x, t, lp, weight=f.double())
    refused(ssv.distill, x, t, lp, grad=torch.zeros((4, 9)))
    refused(ssv.distill, x, t, lp, grad=x.bfloat16())
    refused(ssv.distill, x, t, lp, loss=torch.zeros(5))
    refused(ssv.distill_backward, x, t, lp, torch.zeros((4, 3)))
    refused(ssv.distill_backward, x, t, lp, torch.zeros((4, 4)), grad_loss=torch.zeros(5))


def test_binding_refuses_host_tensors():
    x, tok = torch.zeros((4, 10)), torch.zeros(4, dtype=torch.int32)
    t, lp = torch.zeros((4, 3), dtype=torch.int32), torch.zeros((4, 3))
    for call in (lambda: ssv.logprobs(x, tok, 3), lambda: ssv.distill(x, t, lp, grad=True),
                 lambda: ssv.distill_backward(x, t, lp, torch.zeros((4, 4)))):
        refused(call, match="one CUDA device")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gradients_rows_lie_as_the_logits_do(dtype):
    buf = torch.zeros(4000, dtype=dtype)
    for x in (buf[:300].view(3, 100), buf[1:301].view(3, 100), buf.view(40, 100)[:, :97], buf.view(40, 100)[:, 3:97],
              buf[5:105].view(1, 100)):
        g = ssv._empty_rows(x)
        assert g.shape == x.shape and g.stride(1) == 1
        for i in range(x.shape[0]):
            assert (g[i].data_ptr() - x[i].data_ptr()) % 32 == 0
    wide = ssv._empty_rows(buf.view(4, 1000)[:, :100])
    assert wide.is_contiguous()
